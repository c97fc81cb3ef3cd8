// k_scan.cu -- the gated recurrence over sequences, its gradients and its form for
// single tokens. Per sequence and channel, with gate logits z and s = softplus(-z) / tau,
//     a_t = sigmoid(z_t)^(1/tau) = e^{-s_t},  c_t = 1 - a_t = -expm1(-s_t),
//     h_t = h_{t-1} - c_t h_{t-1} + u_t,      u_t = x_t or c_t x_t (tied).
// The decay is carried as c = 1 - a: with gates near one, 1 - a rounded from a
// would have lost the bits that decide how long the state lasts (a = 1 - 3e-6
// leaves 5 bits of it), and the same error at every step adds up over the
// sequence. Backward, with g_t = dL/dh_t including what the later rows hand down,
//     g_t = dh_t + a_{t+1} g_{t+1},  dx_t = g_t or c_t g_t,
//     dz_t = g_t (h_{t-1} - [tied] x_t) a_t (1 - sigmoid(z_t)) / tau,  dh_0 = a_1 g_1.
// A padded row has c = 0 and u = 0 and is not read.
#include "ops_internal.h"
#include "sm100_ptx.cuh"

namespace msgla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float decay(float z, float inv_tau) {
  const float s = (log1pf(expf(-fabsf(z))) + fmaxf(-z, 0.f)) * inv_tau;
  return -expm1f(-s);
}
// 1 - sigmoid(z)
__device__ __forceinline__ float sigmoid_down(float z) {
  const float e = expf(-fabsf(z));
  return (z >= 0.f ? e : 1.f) / (1.f + e);
}

template <typename T>
__global__ void scan_forward_kernel(const ScanParams p) {
  const int ch = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (ch >= p.D) return;
  const T* x = static_cast<const T*>(p.x.ptr) + b * p.x.batch + ch;
  const T* z = static_cast<const T*>(p.z.ptr) + b * p.z.batch + ch;
  T* o = static_cast<T*>(p.h.ptr) + b * p.h.batch + ch;
  const uint8_t* m = p.mask ? p.mask + static_cast<size_t>(b) * p.L : nullptr;
  const int nsave = (p.L + kScanSave - 1) / kScanSave;
  float h = p.h0 ? p.h0[static_cast<size_t>(b) * p.D + ch] : 0.f;
  for (int t = 0; t < p.L; ++t) {
    if (p.saved && t % kScanSave == 0) p.saved[(static_cast<size_t>(b) * nsave + t / kScanSave) * p.D + ch] = h;
    const bool valid = !m || m[t];
    if (valid) {
      const float c = decay(to_f32(z[t * p.z.row]), p.inv_tau), xv = to_f32(x[t * p.x.row]);
      h = fmaf(-c, h, h) + (p.tied ? c * xv : xv);
    }
    o[t * p.h.row] = from_f32<T>(valid ? h : 0.f);
  }
  p.last[static_cast<size_t>(b) * p.D + ch] = h;
}

template <typename T>
__global__ void scan_backward_kernel(const ScanParams p) {
  const int ch = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (ch >= p.D) return;
  const T* x = static_cast<const T*>(p.x.ptr) + b * p.x.batch + ch;
  const T* z = static_cast<const T*>(p.z.ptr) + b * p.z.batch + ch;
  const T* dh = p.dh.ptr ? static_cast<const T*>(p.dh.ptr) + b * p.dh.batch + ch : nullptr;
  T* dx = static_cast<T*>(p.dx.ptr) + b * p.dx.batch + ch;
  T* dz = static_cast<T*>(p.dz.ptr) + b * p.dz.batch + ch;
  const uint8_t* m = p.mask ? p.mask + static_cast<size_t>(b) * p.L : nullptr;
  const int nsave = (p.L + kScanSave - 1) / kScanSave;
  float carry = p.dlast ? p.dlast[static_cast<size_t>(b) * p.D + ch] : 0.f;
  float before[kScanSave];  // h_{t-1}
  for (int k = nsave - 1; k >= 0; --k) {
    const int t0 = k * kScanSave, n = min(kScanSave, p.L - t0);
    float h = p.saved[(static_cast<size_t>(b) * nsave + k) * p.D + ch];
    for (int r = 0; r < n; ++r) {
      const int t = t0 + r;
      before[r] = h;
      if (m && !m[t]) continue;
      const float c = decay(to_f32(z[t * p.z.row]), p.inv_tau), xv = to_f32(x[t * p.x.row]);
      h = fmaf(-c, h, h) + (p.tied ? c * xv : xv);
    }
    for (int r = n - 1; r >= 0; --r) {
      const int t = t0 + r;
      float vx = 0.f, vz = 0.f;
      if (!m || m[t]) {
        const float zv = to_f32(z[t * p.z.row]), c = decay(zv, p.inv_tau);
        const float g = carry + (dh ? to_f32(dh[t * p.dh.row]) : 0.f);
        vx = p.tied ? c * g : g;
        vz = g * (before[r] - (p.tied ? to_f32(x[t * p.x.row]) : 0.f)) * (1.f - c) * sigmoid_down(zv) * p.inv_tau;
        carry = fmaf(-c, g, g);
      }
      dx[t * p.dx.row] = from_f32<T>(vx);
      dz[t * p.dz.row] = from_f32<T>(vz);
    }
  }
  if (p.dh0) p.dh0[static_cast<size_t>(b) * p.D + ch] = carry;
}

template <typename T>
__global__ void scan_step_kernel(const StepParams p) {
  const int ch = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (ch >= p.D) return;
  float out = 0.f;
  if (!p.mask || p.mask[b]) {
    float* s = p.state + static_cast<size_t>(b) * p.D + ch;
    const float c = decay(to_f32(static_cast<const T*>(p.z)[b * p.z_row + ch]), p.inv_tau);
    const float xv = to_f32(static_cast<const T*>(p.x)[b * p.x_row + ch]), h = *s;
    out = fmaf(-c, h, h) + (p.tied ? c * xv : xv);
    *s = out;
  }
  static_cast<T*>(p.h)[b * p.h_row + ch] = from_f32<T>(out);
}

// f(T{}) with the element type of `dtype`
template <typename F>
void by_dtype(int dtype, F&& f) {
  if (dtype == kBF16) f(__nv_bfloat16{});
  else if (dtype == kF16) f(__half{});
  else f(float{});
}

}  // namespace

cudaError_t launch_scan_forward(const ScanParams& p, cudaStream_t st) {
  const dim3 grid((p.D + 127) / 128, p.B);
  by_dtype(p.dtype, [&](auto t) { scan_forward_kernel<decltype(t)><<<grid, 128, 0, st>>>(p); });
  return cudaGetLastError();
}

cudaError_t launch_scan_backward(const ScanParams& p, cudaStream_t st) {
  const dim3 grid((p.D + 127) / 128, p.B);
  by_dtype(p.dtype, [&](auto t) { scan_backward_kernel<decltype(t)><<<grid, 128, 0, st>>>(p); });
  return cudaGetLastError();
}

cudaError_t launch_scan_step(const StepParams& p, cudaStream_t st) {
  const dim3 grid((p.D + 127) / 128, p.B);
  by_dtype(p.dtype, [&](auto t) { scan_step_kernel<decltype(t)><<<grid, 128, 0, st>>>(p); });
  return cudaGetLastError();
}

}  // namespace msgla
