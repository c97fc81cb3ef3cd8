// k_norm.cu -- group normalisation, channels last, with an activation or an output
// gate, and its gradients. Over the valid rows of one n and the channels of one group,
//     xhat = (x - mean) / sqrt(var + eps)   (no centring: x / sqrt(mean(x^2) + eps)),
//     v = xhat w + b,  y = act(v)  or  v act(gate).
// Backward, with dv = dy act'(v) or dy act(gate), and <.> the mean over the group:
//     dw = sum dv xhat,  db = sum dv,  dgate = dy v act'(gate),
//     dx = (dv w - <dv w> - xhat <dv w xhat>) / sqrt(var + eps)   (no centring: no <dv w>).
// Padded rows enter no sum, give zeros and are not read.
#include "ops_internal.h"
#include "sm100_ptx.cuh"

namespace msgla {
namespace {

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }
__device__ __forceinline__ float act(int kind, float v) {
  return kind == kActNone ? v : kind == kActSilu ? v * sigmoid(v) : sigmoid(v);
}
__device__ __forceinline__ float act_grad(int kind, float v) {
  if (kind == kActNone) return 1.f;
  const float s = sigmoid(v);
  return kind == kActSilu ? s * (1.f + v * (1.f - s)) : s * (1.f - s);
}

constexpr int kThreads = 256;

// Sum of two values over the block, the same in every thread.
__device__ __forceinline__ float2 block_sum(float a, float b) {
  __shared__ float2 part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(~0u, a, o);
    b += __shfl_xor_sync(~0u, b, o);
  }
  __syncthreads();
  if (lane_id() == 0) part[warp_id()] = make_float2(a, b);
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    a += part[i].x;
    b += part[i].y;
  }
  return make_float2(a, b);
}

template <typename T>
__device__ __forceinline__ float value(const Rows& r, long long n, long long s, int c) {
  return to_f32(static_cast<const T*>(r.ptr)[n * r.batch + s * r.row + c]);
}
template <typename T>
__device__ __forceinline__ void put(const Rows& r, long long n, long long s, int c, float v) {
  static_cast<T*>(r.ptr)[n * r.batch + s * r.row + c] = from_f32<T>(v);
}

// One block per (n, group).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormParams p) {
  const long long n = blockIdx.x / p.G;
  const int g = blockIdx.x % p.G, cg = p.C / p.G;
  const long long total = p.S * cg;
  const uint8_t* m = p.mask ? p.mask + n * p.S : nullptr;
  float sum = 0.f, count = 0.f;
  for (long long i = threadIdx.x; i < total; i += kThreads) {
    const long long s = i / cg;
    if (m && !m[s]) continue;
    sum += value<T>(p.x, n, s, g * cg + i % cg);
    count += 1.f;
  }
  const float2 a = block_sum(sum, count);
  const float n_valid = fmaxf(a.y, 1.f), mean = p.center ? a.x / n_valid : 0.f;
  float ss = 0.f;
  for (long long i = threadIdx.x; i < total; i += kThreads) {
    const long long s = i / cg;
    if (m && !m[s]) continue;
    const float d = value<T>(p.x, n, s, g * cg + i % cg) - mean;
    ss += d * d;
  }
  const float rstd = 1.f / sqrtf(block_sum(ss, 0.f).x / n_valid + p.eps);
  if (p.stats && threadIdx.x == 0) {
    p.stats[2 * (n * p.G + g)] = mean;
    p.stats[2 * (n * p.G + g) + 1] = rstd;
  }
  for (long long i = threadIdx.x; i < total; i += kThreads) {
    const long long s = i / cg;
    const int c = g * cg + i % cg;
    float y = 0.f;
    if (!m || m[s]) {
      float v = (value<T>(p.x, n, s, c) - mean) * rstd;
      v = v * (p.w ? p.w[c] : 1.f) + (p.b ? p.b[c] : 0.f);
      y = p.gate.ptr ? v * act(p.act, value<T>(p.gate, n, s, c)) : act(p.act, v);
    }
    put<T>(p.y, n, s, c, y);
  }
}

template <typename T>
__device__ __forceinline__ float grad_v(const NormParams& p, long long n, long long s, int c, float xhat, float& dgate) {
  const float v = xhat * (p.w ? p.w[c] : 1.f) + (p.b ? p.b[c] : 0.f), dy = value<T>(p.dy, n, s, c);
  dgate = 0.f;
  if (!p.gate.ptr) return dy * act_grad(p.act, v);
  const float gv = value<T>(p.gate, n, s, c);
  dgate = dy * v * act_grad(p.act, gv);
  return dy * act(p.act, gv);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormParams p) {
  const long long n = blockIdx.x / p.G;
  const int g = blockIdx.x % p.G, cg = p.C / p.G;
  const long long total = p.S * cg;
  const uint8_t* m = p.mask ? p.mask + n * p.S : nullptr;
  const float mean = p.stats[2 * (n * p.G + g)], rstd = p.stats[2 * (n * p.G + g) + 1];
  float s1 = 0.f, s2 = 0.f, count = 0.f, dg;
  for (long long i = threadIdx.x; i < total; i += kThreads) {
    const long long s = i / cg;
    if (m && !m[s]) continue;
    const int c = g * cg + i % cg;
    const float xhat = (value<T>(p.x, n, s, c) - mean) * rstd;
    const float d = grad_v<T>(p, n, s, c, xhat, dg) * (p.w ? p.w[c] : 1.f);
    s1 += d;
    s2 += d * xhat;
    count += 1.f;
  }
  const float2 a = block_sum(s1, s2);
  const float inv = 1.f / fmaxf(block_sum(count, 0.f).x, 1.f);
  const float m1 = p.center ? a.x * inv : 0.f, m2 = a.y * inv;
  for (long long i = threadIdx.x; i < total; i += kThreads) {
    const long long s = i / cg;
    const int c = g * cg + i % cg;
    float dx = 0.f;
    dg = 0.f;
    if (!m || m[s]) {
      const float xhat = (value<T>(p.x, n, s, c) - mean) * rstd;
      const float d = grad_v<T>(p, n, s, c, xhat, dg) * (p.w ? p.w[c] : 1.f);
      dx = (d - m1 - xhat * m2) * rstd;
    }
    put<T>(p.dx, n, s, c, dx);
    if (p.gate.ptr) put<T>(p.dgate, n, s, c, dg);
  }
}

// One block per channel: dw and db over all rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_weight_kernel(const NormParams p) {
  const int c = blockIdx.x, g = c / (p.C / p.G);
  float s1 = 0.f, s2 = 0.f, dg;
  for (long long i = threadIdx.x; i < p.N * p.S; i += kThreads) {
    const long long n = i / p.S, s = i % p.S;
    if (p.mask && !p.mask[i]) continue;
    const float* st = p.stats + 2 * (n * p.G + g);
    const float xhat = (value<T>(p.x, n, s, c) - st[0]) * st[1], d = grad_v<T>(p, n, s, c, xhat, dg);
    s1 += d * xhat;
    s2 += d;
  }
  const float2 a = block_sum(s1, s2);
  if (threadIdx.x == 0) {
    if (p.dw) p.dw[c] = a.x;
    if (p.db) p.db[c] = a.y;
  }
}

template <typename F>
void by_dtype(int dtype, F&& f) {
  if (dtype == kBF16) f(__nv_bfloat16{});
  else if (dtype == kF16) f(__half{});
  else f(float{});
}

}  // namespace

size_t norm_workspace(const NormParams&, bool) { return 0; }

cudaError_t launch_norm_forward(const NormParams& p, cudaStream_t st) {
  by_dtype(p.dtype, [&](auto t) { norm_forward_kernel<decltype(t)><<<unsigned(p.N * p.G), kThreads, 0, st>>>(p); });
  return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t st) {
  by_dtype(p.dtype, [&](auto t) {
    norm_backward_kernel<decltype(t)><<<unsigned(p.N * p.G), kThreads, 0, st>>>(p);
    if (p.dw || p.db) norm_weight_kernel<decltype(t)><<<p.C, kThreads, 0, st>>>(p);
  });
  return cudaGetLastError();
}

}  // namespace msgla
