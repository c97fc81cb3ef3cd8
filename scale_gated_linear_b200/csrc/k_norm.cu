// k_norm.cu -- group normalisation, channels last, with an activation or an output
// gate, and its gradients. Over the valid rows of one n and the channels of one group,
//     xhat = (x - mean) / sqrt(var + eps)   (no centring: x / sqrt(mean(x^2) + eps)),
//     v = xhat w + b,  y = act(v)  or  v act(gate).
// Backward, with dv = dy act'(v) or dy act(gate), and <.> the mean over the group:
//     dw = sum dv xhat,  db = sum dv,  dgate = dy v act'(gate),
//     dx = (dv w - <dv w> - xhat <dv w xhat>) / sqrt(var + eps)   (no centring: no <dv w>).
// Padded rows enter no sum, give zeros and are not read.
//
// Bound: HBM. Three forms, by shape and alignment:
// * S = 1 and groups of up to 8192 channels: a team of 1 to 32 lanes, or a block, holds one row's
//   group in registers, up to 32 values a lane, so every tensor moves once. Teams keep their channels from row to
//   row: weights stay in registers, and the weight gradients are summed there, joined in
//   shared memory and written once a block. The next row is loaded while one is computed.
// * otherwise, where a sample's rows of a tile of channels fit the shared memory of a cluster of up
//   to eight blocks (1.6 MB in all, and rows aligned to 16 bytes), they are held there: every tensor moves
//   once here too;
// * else two passes over blocks of rows and channels: sums first, then the result, which
//   reads x (and dy) again, from L2 where a pass fits there.
// Measured, bf16: 65536 groups of 512 (16384 x 2048) under an output gate forward 37 us (82 % of copy
// bandwidth), backward 73 and 6 for the weights (70 %); 8 x 2048 x 1024 in 32 groups with padding
// 78 us forward and backward held in shared memory, 97 in two passes.
// Variances are sums of squared differences: from the mean itself in registers; held, from a mean that
// the sum of the differences corrects; in two passes from each thread's first value, joined by count, mean and
// sum of squares. So a mean far from zero costs what rounding it to f32 costs (in registers, the few additions
// of a row's team too). Everything is summed in f32 in a fixed order.
#include <type_traits>

#include "ops_internal.h"
#include "sm100_ptx.cuh"

namespace msgla {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(-kLog2e * v)));
  return r;
}
// act(v), and with it act'(v)
template <int KIND>
__device__ __forceinline__ float act(float v) {
  if (KIND == kActNone) return v;
  const float s = sigmoid(v);
  return KIND == kActSilu ? v * s : s;
}
template <int KIND>
__device__ __forceinline__ float2 act_both(float v) {
  if (KIND == kActNone) return make_float2(v, 1.f);
  const float s = sigmoid(v);
  if (KIND == kActSilu) return make_float2(v * s, fmaf(v * s, 1.f - s, s));
  return make_float2(s, s * (1.f - s));
}
// f(activation, gated) with the values as compile-time constants: one branch for a row or a
// block's rows in place of one an element.
template <int N>
struct Const {
  __host__ __device__ constexpr operator int() const { return N; }
};
template <typename F>
__device__ __forceinline__ void by_act(int kind, bool gated, F&& f) {
  auto with = [&](auto k) {
    if (gated) f(k, Const<1>{});
    else f(k, Const<0>{});
  };
  if (kind == kActNone) with(Const<kActNone>{});
  else if (kind == kActSilu) with(Const<kActSilu>{});
  else with(Const<kActSigmoid>{});
}

// V neighbouring channels as loaded: 16 bytes, or one element where rows are not aligned to 16.
template <typename T, int V>
struct Vec {
  uint32_t w[V == 1 ? 1 : 4];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> zeros() {
  Vec<T, V> r;
#pragma unroll
  for (uint32_t& w : r.w) w = 0;
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  Vec<T, V> r;
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 4) r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    else r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else {
    static_assert(V * sizeof(T) == 16, "16 bytes");
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const Vec<T, V>& r) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(p) = r.w[0];
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(r.w[0]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
}
// The two 16-bit values of a word as f32, and back.
template <typename T>
__device__ __forceinline__ float2 pair_f32(uint32_t w) {
  if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pair_round(float a, float b) {
  if constexpr (std::is_same_v<T, __half>) return pack_half2(a, b);
  else return pack_bf162(a, b);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& r, float (&f)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = __uint_as_float(r.w[e]);
  } else if constexpr (V == 1) {
    f[0] = pair_f32<T>(r.w[0]).x;
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 v = pair_f32<T>(r.w[e / 2]);
      f[e] = v.x, f[e + 1] = v.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
  Vec<T, V> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) r.w[e] = __float_as_uint(f[e]);
  } else if constexpr (V == 1) {
    r.w[0] = pair_round<T>(f[0], 0.f);
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) r.w[e / 2] = pair_round<T>(f[e], f[e + 1]);
  }
  return r;
}

// V weights from channel c on (16-byte loads where V allows), or `none` without weights
template <int V>
__device__ __forceinline__ void weights(const float* w, int c, bool in, float none, float (&to)[V]) {
  if (!w || !in) {
#pragma unroll
    for (int e = 0; e < V; ++e) to[e] = none;
  } else if constexpr (V == 1) {
    to[0] = __ldg(w + c);
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(w + c + e));
      to[e] = f.x, to[e + 1] = f.y, to[e + 2] = f.z, to[e + 3] = f.w;
    }
  }
}
template <typename T>
__device__ __forceinline__ T* at(const Rows& r, long long n, long long s, int c) {
  return static_cast<T*>(r.ptr) + n * r.batch + s * r.row + c;
}

__device__ __forceinline__ float team_sum(float v, int team) {
  for (int o = team >> 1; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// N sums over a team of TEAM threads (0: `team`, below 32). A whole block's go through `part`,
// two buffers taken in turn so that one barrier a call is enough.
template <int TEAM, int N>
__device__ __forceinline__ void sums_of(float (&v)[N], int team, float (*part)[2][kThreads / 32], int turn) {
  if constexpr (TEAM == 0) {
    for (int o = team >> 1; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  }
  if constexpr (TEAM == kThreads) {
    if (lane_id() == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) part[turn][k][warp_id()] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) v[k] += part[turn][k][i];
    }
  }
}

// Gradient of the value before the activation, and of the gate.
template <int KIND, bool GATED>
__device__ __forceinline__ float grad_v(float v, float dy, float gate, float& dgate) {
  if (!GATED) {
    dgate = 0.f;
    return dy * act_both<KIND>(v).y;
  }
  const float2 a = act_both<KIND>(gate);
  dgate = dy * v * a.y;
  return dy * a.x;
}

// ---------------------------------------------------------------- S = 1: rows in registers
// Block (slice, y): `gs` groups from slice * gs on, rows (y + k * gridDim.y) * rpi + team / gs.
struct RowPlan {
  int team, gs, rpi, slices, blocks;  // threads of a team, groups and rows a block, grid
};

template <typename T, int V, int NV>
struct RowLane {
  int c, step;  // first channel, channels between two vectors
  int g, row;   // group, and the first row
  int vectors;  // how many of the NV exist
  __device__ __forceinline__ RowLane(const NormParams& p, const RowPlan& q) {
    const int team = threadIdx.x / q.team, tl = threadIdx.x % q.team, cg = p.C / p.G;
    g = blockIdx.x * q.gs + team % q.gs;
    row = team / q.gs;
    step = q.team * V;
    c = g * cg + tl * V;
    vectors = row < q.rpi && g < p.G && tl * V < cg ? (cg - tl * V + step - 1) / step : 0;
  }
  __device__ __forceinline__ bool in(int i) const { return i < vectors; }
};
// A lane's vectors of the rows it takes one after another.
template <typename T, int V>
struct RowPtr {
  T* at;
  long long step;
  __device__ __forceinline__ RowPtr(const Rows& r, long long row, long long rows, int c) {
    at = r.ptr ? static_cast<T*>(r.ptr) + row * r.batch + c : nullptr;
    step = rows * r.batch;
  }
};

template <typename T, int V, int NV, int TEAM>
__global__ void __launch_bounds__(kThreads, V * NV <= 16 ? 3 : 1) norm_rows_forward_kernel(const NormParams p, const RowPlan q) {
  __shared__ float part[2][2][kThreads / 32];
  const RowLane<T, V, NV> l(p, q);
  const float inv = 1.f / (p.C / p.G);
  const bool gated = p.gate.ptr;
  const long long step = static_cast<long long>(gridDim.y) * q.rpi;
  long long base = static_cast<long long>(blockIdx.y) * q.rpi, row = base + l.row;
  RowPtr<T, V> px(p.x, row, step, l.c), pg(p.gate, row, step, l.c), py(p.y, row, step, l.c);
  Vec<T, V> xn[NV], gn[NV];
  bool valid_next;
  auto fetch = [&](long long r) {
    valid_next = r < p.N && (!p.mask || p.mask[r]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xn[i] = valid_next && l.in(i) ? load<T, V>(px.at + i * l.step) : zeros<T, V>();
      gn[i] = valid_next && l.in(i) && gated ? load<T, V>(pg.at + i * l.step) : zeros<T, V>();
    }
    px.at += px.step;
    pg.at += pg.step;
  };
  fetch(row);
  for (; base < p.N; base += step, row += step, py.at += py.step) {
    float x[NV][V], sum[1] = {0.f}, ss[1] = {0.f};
    Vec<T, V> gt[NV];
    const bool valid = valid_next;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      gt[i] = gn[i];
      unpack(xn[i], x[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum[0] += x[i][e];
    }
    if (base + step < p.N) fetch(row + step);
    if (p.center) sums_of<TEAM>(sum, q.team, part, 0);
    const float mean = p.center ? sum[0] * inv : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float off = l.in(i) ? mean : 0.f;  // what does not exist stays zero
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i][e] -= off;
        ss[0] = fmaf(x[i][e], x[i][e], ss[0]);
      }
    }
    sums_of<TEAM>(ss, q.team, part, 1);
    const float rstd = 1.f / sqrtf(ss[0] * inv + p.eps);
    if (TEAM == kThreads && !p.center) __syncthreads();  // the next row writes the same buffer
    if (row >= p.N) continue;
    if (p.stats && l.vectors && threadIdx.x % q.team == 0)
      *reinterpret_cast<float2*>(p.stats + 2 * (row * p.G + l.g)) = make_float2(mean, rstd);
    if (!valid) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (l.in(i)) store<T, V>(py.at + i * l.step, zeros<T, V>());
      continue;
    }
    by_act(p.act, gated, [&](auto kind, auto with_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!l.in(i)) continue;
        float w[V], b[V], g[V], y[V];
        weights<V>(p.w, l.c + i * l.step, true, 1.f, w);
        weights<V>(p.b, l.c + i * l.step, true, 0.f, b);
        if (with_gate) unpack(gt[i], g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = fmaf(x[i][e] * rstd, w[e], b[e]);
          y[e] = with_gate ? v * act<kind>(g[e]) : act<kind>(v);
        }
        store<T, V>(py.at + i * l.step, pack<T, V>(y));
      }
    });
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Weight gradients: partial sums [blocks][2][C] (dw, db) in the workspace. Rows come through
// shared memory, two ahead, each lane copying what it reads itself: held in registers, the
// next row's 24 words beside the sums' 32 were moved behind the arithmetic or spilled (123 us
// where this takes 73, at 65536 groups of 512).
constexpr int kAhead = 2;
template <typename T, int V, int NV>
constexpr int kRowStage = kThreads * NV * 3 * (V == 1 ? 4 : 16);  // bytes of a block's rows

template <typename T, int V, int NV, int TEAM>
__global__ void __launch_bounds__(kThreads, V * NV <= 16 ? 2 : 1) norm_rows_backward_kernel(const NormParams p, const RowPlan q) {
  __shared__ float part[2][2][kThreads / 32];
  griddep_launch();
  extern __shared__ __align__(16) uint8_t dynamic[];  // rows; in the end [rpi - 1][gs * cg][2] sums
  constexpr bool kKeep = V * NV <= 16;  // weights in registers
  int turn = 0;
  const RowLane<T, V, NV> l(p, q);
  const int cg = p.C / p.G;
  const float inv = 1.f / cg;
  const bool gated = p.gate.ptr;
  float dw[NV][V] = {}, db[NV][V] = {}, w[kKeep ? NV : 1][V], b[kKeep ? NV : 1][V];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      weights<V>(p.w, l.c + i * l.step, l.in(i), 1.f, w[i]);
      weights<V>(p.b, l.c + i * l.step, l.in(i), 0.f, b[i]);
    }
  }
  const long long step = static_cast<long long>(gridDim.y) * q.rpi;
  long long base = static_cast<long long>(blockIdx.y) * q.rpi, row = base + l.row, coming = row;
  RowPtr<T, V> px(p.x, row, step, l.c), pd(p.dy, row, step, l.c), pg(p.gate, row, step, l.c), ox(p.dx, row, step, l.c),
      og(p.dgate, row, step, l.c);
  const float2* stats = reinterpret_cast<const float2*>(p.stats) + row * p.G + l.g;
  const long long stat_step = step * p.G;
  // vector i of tensor k of stage s: kThreads neighbouring words or quadruples
  using Word = std::conditional_t<V == 1, uint32_t, uint4>;
  Word* mine = reinterpret_cast<Word*>(dynamic) + threadIdx.x;
  auto slot = [&](int s, int k, int i) { return mine + ((s * 3 + k) * NV + i) * kThreads; };
  float2 st_next[kAhead];
  uint32_t valid_bits = 0;
  auto fetch = [&](int s) {
    const bool valid = coming < p.N && l.vectors && (!p.mask || p.mask[coming]);
    valid_bits = valid ? valid_bits | 1u << s : valid_bits & ~(1u << s);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const T* from = k == 0 ? px.at : k == 1 ? pd.at : pg.at;
      if (k == 2 && !gated) break;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Word* to = slot(s, k, i);
        if constexpr (V == 1) {
          *to = valid && l.in(i) ? load<T, V>(from + i * l.step).w[0] : 0u;
        } else {
          if (valid && l.in(i)) copy16(smem_u32(to), from + i * l.step);
          else *to = make_uint4(0, 0, 0, 0);
        }
      }
    }
    copies_commit();
    const float2 got = valid ? *stats : make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j == s) st_next[j] = got;
    px.at += px.step;
    pd.at += pd.step;
    pg.at += pg.step;
    stats += stat_step;
    coming += step;
  };
  auto read = [&](int s, int k, int i, float (&f)[V]) {
    Vec<T, V> v;
    if constexpr (V == 1) {
      v.w[0] = *slot(s, k, i);
    } else {
      const uint4 u = *slot(s, k, i);
      v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    }
    unpack(v, f);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) fetch(s);
  int s = 0;
  for (; base < p.N; base += step, row += step, ox.at += ox.step, og.at += og.step) {
    copies_wait<kAhead - 1>();
    float2 st = st_next[0];
#pragma unroll
    for (int j = 1; j < kAhead; ++j)
      if (j == s) st = st_next[j];
    const bool valid = valid_bits >> s & 1, here = row < p.N;
    float sums[2] = {0.f, 0.f}, dv[NV][V], xh[NV][V];
    by_act(p.act, gated, [&](auto kind, auto with_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float dy[V], gv[V], dg[V], wl[V], bl[V];
        if constexpr (!kKeep) {
          weights<V>(p.w, l.c + i * l.step, l.in(i), 1.f, wl);
          weights<V>(p.b, l.c + i * l.step, l.in(i), 0.f, bl);
        }
        read(s, 0, i, xh[i]);
        read(s, 1, i, dy);
        if (with_gate) read(s, 2, i, gv);
#pragma unroll
        for (int e = 0; e < V; ++e) {  // where nothing was loaded dy = 0, and with it every sum's part
          const float we = kKeep ? w[kKeep ? i : 0][e] : wl[e], be = kKeep ? b[kKeep ? i : 0][e] : bl[e];
          xh[i][e] = (xh[i][e] - st.x) * st.y;
          const float t = grad_v<kind, with_gate>(fmaf(xh[i][e], we, be), dy[e], with_gate ? gv[e] : 0.f, dg[e]);
          dw[i][e] = fmaf(t, xh[i][e], dw[i][e]);
          db[i][e] += t;
          dv[i][e] = t * we;
          sums[0] += dv[i][e];
          sums[1] = fmaf(dv[i][e], xh[i][e], sums[1]);
        }
        if (with_gate && here && l.in(i)) store<T, V>(og.at + i * l.step, pack<T, V>(dg));
      }
    });
    fetch(s);
    s = s + 1 == kAhead ? 0 : s + 1;
    sums_of<TEAM>(sums, q.team, part, turn ^= 1);
    const float m1 = p.center ? sums[0] * inv : 0.f, m2 = sums[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dx[V];
#pragma unroll
      for (int e = 0; e < V; ++e) dx[e] = (dv[i][e] - m1 - xh[i][e] * m2) * st.y;
      if (here && l.in(i)) store<T, V>(ox.at + i * l.step, valid ? pack<T, V>(dx) : zeros<T, V>());
    }
  }
  if (!p.dw && !p.db) return;
  // the block's rows of every channel, summed in order by the first one's team
  copies_wait<0>();
  __syncthreads();
  float* shared = reinterpret_cast<float*>(dynamic);
  const int width = q.gs * cg, c0 = blockIdx.x * width;
  if (l.row > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (l.in(i))
#pragma unroll
        for (int e = 0; e < V; ++e)
          *reinterpret_cast<float2*>(shared + 2 * ((l.row - 1) * width + l.c + i * l.step + e - c0)) = make_float2(dw[i][e], db[i][e]);
  }
  __syncthreads();
  if (l.row > 0) return;
  float* out = static_cast<float*>(p.workspace) + static_cast<size_t>(blockIdx.y) * 2 * p.C;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (l.in(i))
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = l.c + i * l.step + e;
        float2 s = make_float2(dw[i][e], db[i][e]);
        for (int r = 1; r < q.rpi; ++r) {
          const float2 o = *reinterpret_cast<const float2*>(shared + 2 * ((r - 1) * width + c - c0));
          s.x += o.x;
          s.y += o.y;
        }
        out[c] = s.x;
        out[p.C + c] = s.y;
      }
}

// dw and db from `rows` partial sums [rows][2][C]. 32 channels a block.
__global__ void __launch_bounds__(1024) norm_weights_kernel(const NormParams p, const float* part, int rows) {
  __shared__ float2 sums[32][33];
  griddep_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float2 s = make_float2(0.f, 0.f);
  if (c < p.C)
    for (int r = threadIdx.y; r < rows; r += 32) {
      const float* f = part + static_cast<size_t>(r) * 2 * p.C + c;
      s.x += f[0];
      s.y += f[p.C];
    }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = sums[threadIdx.x][threadIdx.y];  // the 32 partial sums of one channel, in one warp
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s.x += __shfl_xor_sync(~0u, s.x, o);
    s.y += __shfl_xor_sync(~0u, s.y, o);
  }
  const int co = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && co < p.C) {
    if (p.dw) p.dw[co] = s.x;
    if (p.db) p.db[co] = s.y;
  }
}

// ---------------------------------------------------------------- blocks of rows and channels
// Block (n, chunk, tile): `ty` rows at a time of tx vectors of channels. Workspace: per (n,
// chunk) and segment (the part of group g inside tile t, number g + t of at most groups + tiles)
// two numbers; with gradients also per channel.
struct BlockPlan {
  int tx, ty, width;  // threads along channels and rows, channels a tile
  int tiles, chunks, rows;  // rows a chunk
  int segments;             // groups + tiles
};

struct Part {
  long long n;
  int chunk, tile;
  __device__ __forceinline__ explicit Part(const BlockPlan& q) {
    unsigned i = blockIdx.x;
    tile = i % q.tiles;
    i /= q.tiles;
    chunk = i % q.chunks;
    n = i / q.chunks;
  }
};

constexpr int kUnroll = 4;  // rows a thread has on their way at once
// Valid rows among s, s + ty, .. s + 3 ty (bit k: the k-th).
__device__ __forceinline__ uint32_t rows_valid(const uint8_t* m, long long s, long long s1, int ty) {
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (s + k * ty < s1 && (!m || m[s + k * ty])) bits |= 1u << k;
  return bits;
}

// Forward sums: float2 (mean, sum of squared differences) per segment at
// seg[(n * chunks + chunk) * segments + segment]; the valid rows of each (n, chunk) at rows_of.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_sums_kernel(const NormParams p, const BlockPlan q, float2* seg, float* rows_of) {
  __shared__ float2 cell[kThreads];  // a thread's V channels: mean and squares
  __shared__ int counts[kThreads];
  griddep_launch();
  const Part part(q);
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx, c = part.tile * q.width + tx * V, cg = p.C / p.G;
  const long long s0 = static_cast<long long>(part.chunk) * q.rows, s1 = min(s0 + q.rows, p.S);
  const uint8_t* m = p.mask ? p.mask + part.n * p.S : nullptr;
  float first = 0.f, sum[V] = {}, sq[V] = {};
  int count = 0;
  if (c < p.C) {
    const T* x = at<T>(p.x, part.n, 0, c);
    long long s = s0 + ty;
    if (p.center) {  // differences from the thread's first value
      while (s < s1 && m && !m[s]) s += q.ty;
      if (s < s1) first = to_f32(x[s * p.x.row]);
    }
    uint32_t next = rows_valid(m, s, s1, q.ty);
    for (; s < s1; s += kUnroll * q.ty) {
      const uint32_t bits = next;
      Vec<T, V> v[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (bits >> k & 1) v[k] = load<T, V>(x + (s + k * q.ty) * p.x.row);
      next = rows_valid(m, s + kUnroll * q.ty, s1, q.ty);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (bits >> k & 1) {
          float f[V];
          unpack(v[k], f);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float d = f[e] - first;
            sum[e] += d;
            sq[e] = fmaf(d, d, sq[e]);
          }
        }
      count += __popc(bits);
    }
  }
  // the V channels are of one group: about their common mean
  float total = 0.f, squares = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) total += sum[e];
  const float n = static_cast<float>(max(count, 1)), off = p.center ? total / (n * V) : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float own = sum[e] / n;  // sum (d - off)^2 = sum (d - own)^2 + n (own - off)^2
    squares += p.center ? fmaxf(sq[e] - sum[e] * own, 0.f) + n * (own - off) * (own - off) : sq[e];
  }
  cell[threadIdx.x] = make_float2(first + off, squares);
  if (tx == 0) counts[ty] = count;
  __syncthreads();
  int rows = 0;
  for (int r = 0; r < q.ty; ++r) rows += counts[r];
  if (part.tile == 0 && threadIdx.x == 0) rows_of[part.n * q.chunks + part.chunk] = static_cast<float>(rows);
  // one warp joins a segment: its mean, then the squares about it
  const int t0 = part.tile * q.width, t1 = min(t0 + q.width, p.C);
  for (int g = t0 / cg + warp_id(); g * cg < t1; g += kThreads / 32) {
    const int a = max(g * cg, t0), x0 = (a - t0) / V, wide = (min((g + 1) * cg, t1) - a) / V, cells = wide * q.ty;
    float sums = 0.f, sqs = 0.f, mean = 0.f;
    if (p.center && rows) {
      int r0 = 0;
      while (counts[r0] == 0) ++r0;
      const float base = cell[r0 * q.tx + x0].x;
      for (int i = lane_id(); i < cells; i += 32) {
        const int r = i / wide;
        if (counts[r]) sums += counts[r] * (cell[r * q.tx + x0 + i - r * wide].x - base);
      }
      mean = base + team_sum(sums, 32) / (static_cast<float>(rows) * wide);
    }
    for (int i = lane_id(); i < cells; i += 32) {
      const int r = i / wide;
      if (!counts[r]) continue;
      const float2 v = cell[r * q.tx + x0 + i - r * wide];
      const float d = v.x - mean;
      sqs += v.y + counts[r] * V * d * d;
    }
    sqs = team_sum(sqs, 32);
    if (lane_id() == 0) seg[(part.n * q.chunks + part.chunk) * q.segments + g + part.tile] = make_float2(mean, sqs);
  }
}

// Count, mean and sum of squared differences of two sets joined.
struct Moments {
  float n, mean, squares;
  __device__ __forceinline__ void join(float m, float mu, float sq) {
    if (m <= 0.f) return;
    const float all = n + m, d = mu - mean, share = m / all;
    mean = n > 0.f ? fmaf(d, share, mean) : mu;
    squares += sq + (n > 0.f ? d * d * n * share : 0.f);
    n = all;
  }
};
// Joins the segments of group g of sample n (one warp): mean and 1 / sqrt(var + eps), in lane 0.
__device__ __forceinline__ float2 join_stats(const NormParams& p, const BlockPlan& q, long long n, int g, const float2* seg,
                                             const float* rows_of) {
  const int cg = p.C / p.G, a = g * cg, t0 = a / q.width, segs = (a + cg - 1) / q.width - t0 + 1;
  Moments m{0.f, 0.f, 0.f};
  for (int i = lane_id(); i < segs * q.chunks; i += 32) {
    const int chunk = i / segs, t = t0 + i % segs, lo = max(a, t * q.width), hi = min(a + cg, (t + 1) * q.width);
    const float2 v = seg[(n * q.chunks + chunk) * q.segments + g + t];
    m.join(rows_of[n * q.chunks + chunk] * (hi - lo), v.x, v.y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float k = __shfl_down_sync(~0u, m.n, o), mu = __shfl_down_sync(~0u, m.mean, o), sq = __shfl_down_sync(~0u, m.squares, o);
    m.join(k, mu, sq);
  }
  return make_float2(p.center ? m.mean : 0.f, 1.f / sqrtf(m.squares / fmaxf(m.n, 1.f) + p.eps));
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) norm_apply_kernel(const NormParams p, const BlockPlan q, const float2* seg,
                                                              const float* rows_of) {
  extern __shared__ float2 stat[];  // groups that meet the tile
  griddep_launch();
  const Part part(q);
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx, c = part.tile * q.width + tx * V, cg = p.C / p.G;
  const int t0 = part.tile * q.width, t1 = min(t0 + q.width, p.C), g0 = t0 / cg;
  griddep_wait();
  for (int g = g0 + warp_id(); g * cg < t1; g += kThreads / 32) {
    const float2 v = join_stats(p, q, part.n, g, seg, rows_of);
    if (lane_id() == 0) {
      stat[g - g0] = v;
      if (p.stats && part.chunk == 0 && g * cg >= t0) *reinterpret_cast<float2*>(p.stats + 2 * (part.n * p.G + g)) = v;
    }
  }
  __syncthreads();
  if (c >= p.C) return;
  const float2 st = stat[c / cg - g0];  // a vector's channels are of one group
  float w[V], b[V];
  weights<V>(p.w, c, true, 1.f, w);
  weights<V>(p.b, c, true, 0.f, b);
#pragma unroll
  for (int e = 0; e < V; ++e) w[e] *= st.y;
  const long long s0 = static_cast<long long>(part.chunk) * q.rows, s1 = min(s0 + q.rows, p.S);
  const uint8_t* m = p.mask ? p.mask + part.n * p.S : nullptr;
  const T* xp = at<T>(p.x, part.n, 0, c);
  const T* gp = at<T>(p.gate, part.n, 0, c);
  T* yp = at<T>(p.y, part.n, 0, c);
  by_act(p.act, p.gate.ptr, [&](auto kind, auto gated) {
    uint32_t next = rows_valid(m, s0 + ty, s1, q.ty);
    for (long long s = s0 + ty; s < s1; s += kUnroll * q.ty) {
      const uint32_t bits = next;
      Vec<T, V> x[kUnroll], gt[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (bits >> k & 1) {
          x[k] = load<T, V>(xp + (s + k * q.ty) * p.x.row);
          if (gated) gt[k] = load<T, V>(gp + (s + k * q.ty) * p.gate.row);
        }
      next = rows_valid(m, s + kUnroll * q.ty, s1, q.ty);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        Vec<T, V> y = zeros<T, V>();
        if (bits >> k & 1) {
          float xv[V], gv[V], r[V];
          unpack(x[k], xv);
          if (gated) unpack(gt[k], gv);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float v = fmaf(xv[e] - st.x, w[e], b[e]);
            r[e] = gated ? v * act<kind>(gv[e]) : act<kind>(v);
          }
          y = pack<T, V>(r);
        }
        if (s + k * q.ty < s1) store<T, V>(yp + (s + k * q.ty) * p.y.row, y);
      }
    }
  });
}

// Backward sums: per channel dw and db of every (n, chunk) as chan[(n * chunks + chunk)][2][C], per
// segment (sum dv w, sum dv w xhat) as seg, and the valid rows.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) norm_grad_sums_kernel(const NormParams p, const BlockPlan q, float* chan, float2* seg,
                                                                  float* rows_of) {
  extern __shared__ float2 cell[];  // [ty][width]
  __shared__ int counts[kThreads];
  griddep_launch();
  const Part part(q);
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx, c = part.tile * q.width + tx * V, cg = p.C / p.G;
  const long long s0 = static_cast<long long>(part.chunk) * q.rows, s1 = min(s0 + q.rows, p.S);
  const uint8_t* m = p.mask ? p.mask + part.n * p.S : nullptr;
  const size_t at_part = static_cast<size_t>(part.n) * q.chunks + part.chunk;
  float w[V], b[V], dw[V] = {}, db[V] = {};
  int count = 0;
  if (c < p.C) {
    const float2 st = *reinterpret_cast<const float2*>(p.stats + 2 * (part.n * p.G + c / cg));
    weights<V>(p.w, c, true, 1.f, w);
    weights<V>(p.b, c, true, 0.f, b);
    const T* xp = at<T>(p.x, part.n, 0, c);
    const T* dp = at<T>(p.dy, part.n, 0, c);
    const T* gp = at<T>(p.gate, part.n, 0, c);
    by_act(p.act, p.gate.ptr, [&](auto kind, auto gated) {
      uint32_t next = rows_valid(m, s0 + ty, s1, q.ty);
      for (long long s = s0 + ty; s < s1; s += kUnroll * q.ty) {
        const uint32_t bits = next;
        count += __popc(bits);
        Vec<T, V> x[kUnroll], d[kUnroll], gt[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
          if (bits >> k & 1) {
            x[k] = load<T, V>(xp + (s + k * q.ty) * p.x.row);
            d[k] = load<T, V>(dp + (s + k * q.ty) * p.dy.row);
            if (gated) gt[k] = load<T, V>(gp + (s + k * q.ty) * p.gate.row);
          }
        next = rows_valid(m, s + kUnroll * q.ty, s1, q.ty);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
          if (bits >> k & 1) {
            float xv[V], dy[V], gv[V], dg;
            unpack(x[k], xv);
            unpack(d[k], dy);
            if (gated) unpack(gt[k], gv);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float xh = (xv[e] - st.x) * st.y;
              const float t = grad_v<kind, gated>(fmaf(xh, w[e], b[e]), dy[e], gated ? gv[e] : 0.f, dg);
              dw[e] = fmaf(t, xh, dw[e]);
              db[e] += t;
            }
          }
      }
    });
#pragma unroll
    for (int e = 0; e < V; ++e) cell[ty * q.width + tx * V + e] = make_float2(dw[e], db[e]);
  }
  if (tx == 0) counts[ty] = count;
  __syncthreads();
  if (part.tile == 0 && threadIdx.x == 0) {
    int rows = 0;
    for (int r = 0; r < q.ty; ++r) rows += counts[r];
    rows_of[at_part] = static_cast<float>(rows);
  }
  const int t0 = part.tile * q.width, t1 = min(t0 + q.width, p.C);
  for (int i = threadIdx.x; i < t1 - t0; i += kThreads) {
    float2 s = cell[i];
    for (int r = 1; r < q.ty; ++r) {
      s.x += cell[r * q.width + i].x;
      s.y += cell[r * q.width + i].y;
    }
    if (p.dw || p.db) {
      chan[at_part * 2 * p.C + t0 + i] = s.x;
      chan[at_part * 2 * p.C + p.C + t0 + i] = s.y;
    }
    const float wi = p.w ? p.w[t0 + i] : 1.f;
    cell[i] = make_float2(s.y * wi, s.x * wi);
  }
  __syncthreads();
  for (int g = t0 / cg + warp_id(); g * cg < t1; g += kThreads / 32) {
    const int a = max(g * cg, t0), wide = min((g + 1) * cg, t1) - a;
    float s1v = 0.f, s2v = 0.f;
    for (int i = lane_id(); i < wide; i += 32) {
      s1v += cell[a - t0 + i].x;
      s2v += cell[a - t0 + i].y;
    }
    s1v = team_sum(s1v, 32);
    s2v = team_sum(s2v, 32);
    if (lane_id() == 0) seg[at_part * q.segments + g + part.tile] = make_float2(s1v, s2v);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) norm_grad_apply_kernel(const NormParams p, const BlockPlan q, const float2* seg,
                                                                   const float* rows_of) {
  extern __shared__ float2 stat[];  // <dv w>, <dv w xhat> of the groups that meet the tile
  griddep_launch();
  const Part part(q);
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx, c = part.tile * q.width + tx * V, cg = p.C / p.G;
  const int t0 = part.tile * q.width, t1 = min(t0 + q.width, p.C), g0 = t0 / cg;
  griddep_wait();
  for (int g = g0 + warp_id(); g * cg < t1; g += kThreads / 32) {
    const int a = g * cg, first = a / q.width, segs = (a + cg - 1) / q.width - first + 1;
    float s1v = 0.f, s2v = 0.f, count = 0.f;
    for (int i = lane_id(); i < segs * q.chunks; i += 32) {
      const size_t row = static_cast<size_t>(part.n) * q.chunks + i / segs;
      const float2 v = seg[row * q.segments + g + first + i % segs];
      s1v += v.x;
      s2v += v.y;
      if (i % segs == 0) count += rows_of[row];
    }
    s1v = team_sum(s1v, 32);
    s2v = team_sum(s2v, 32);
    count = fmaxf(team_sum(count, 32), 1.f) * cg;
    if (lane_id() == 0) stat[g - g0] = make_float2(p.center ? s1v / count : 0.f, s2v / count);
  }
  __syncthreads();
  if (c >= p.C) return;
  const float2 st = *reinterpret_cast<const float2*>(p.stats + 2 * (part.n * p.G + c / cg)), mm = stat[c / cg - g0];
  float w[V], b[V];
  weights<V>(p.w, c, true, 1.f, w);
  weights<V>(p.b, c, true, 0.f, b);
  const long long s0 = static_cast<long long>(part.chunk) * q.rows, s1 = min(s0 + q.rows, p.S);
  const uint8_t* m = p.mask ? p.mask + part.n * p.S : nullptr;
  const T* xp = at<T>(p.x, part.n, 0, c);
  const T* dp = at<T>(p.dy, part.n, 0, c);
  const T* gp = at<T>(p.gate, part.n, 0, c);
  T* ox = at<T>(p.dx, part.n, 0, c);
  T* og = at<T>(p.dgate, part.n, 0, c);
  by_act(p.act, p.gate.ptr, [&](auto kind, auto gated) {
    uint32_t next = rows_valid(m, s0 + ty, s1, q.ty);
    for (long long s = s0 + ty; s < s1; s += kUnroll * q.ty) {
      const uint32_t bits = next;
      Vec<T, V> x[kUnroll], d[kUnroll], gt[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (bits >> k & 1) {
          x[k] = load<T, V>(xp + (s + k * q.ty) * p.x.row);
          d[k] = load<T, V>(dp + (s + k * q.ty) * p.dy.row);
          if (gated) gt[k] = load<T, V>(gp + (s + k * q.ty) * p.gate.row);
        }
      next = rows_valid(m, s + kUnroll * q.ty, s1, q.ty);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        Vec<T, V> dx = zeros<T, V>(), dgate = dx;
        if (bits >> k & 1) {
          float xv[V], dy[V], gv[V], dg[V], r[V];
          unpack(x[k], xv);
          unpack(d[k], dy);
          if (gated) unpack(gt[k], gv);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float xh = (xv[e] - st.x) * st.y;
            const float t = grad_v<kind, gated>(fmaf(xh, w[e], b[e]), dy[e], gated ? gv[e] : 0.f, dg[e]) * w[e];
            r[e] = (t - mm.x - xh * mm.y) * st.y;
          }
          dx = pack<T, V>(r);
          if (gated) dgate = pack<T, V>(dg);
        }
        if (s + k * q.ty < s1) {
          store<T, V>(ox + (s + k * q.ty) * p.dx.row, dx);
          if (gated) store<T, V>(og + (s + k * q.ty) * p.dgate.row, dgate);
        }
      }
    }
  });
}

// ---------------------------------------------------------------- samples held in shared memory
// A cluster of blocks holds a sample's rows of one tile (whole groups of channels) in shared memory:
// x, or x, dy and gate, are read from HBM once, and the group sums pass between the blocks through
// distributed shared memory. A thread copies and uses the same 16-byte vectors throughout,
// so only sums and valid rows need barriers.
struct HoldPlan {
  int cluster, rows;      // blocks a sample and tile, rows a block
  int tx, ty, width;      // vectors along the tile, rows at once, channels
  int tiles, groups;      // tiles, groups a tile
  int shared;             // bytes
};
constexpr int kMaxHold = 8;
constexpr int kHoldShared = 212 * 1024;  // most that a block asks for

template <typename T, int V, int TENSORS>
struct Hold {
  uint4* data;       // [tensor][row][tx]
  float2* red;       // [kThreads]
  float2* slots;     // [2][cluster][groups + 1], written by the cluster's blocks
  uint8_t* valid;    // [rows]
  const HoldPlan& q;
  int rank, tx, ty, c, tile, rows;
  long long n, s0;
  bool here;         // the thread has a vector
  __device__ __forceinline__ Hold(const NormParams& p, const HoldPlan& plan, uint8_t* dynamic) : q(plan) {
    data = reinterpret_cast<uint4*>(dynamic);
    red = reinterpret_cast<float2*>(data + static_cast<size_t>(TENSORS) * q.rows * q.tx);
    slots = red + kThreads;
    valid = reinterpret_cast<uint8_t*>(slots + 2 * q.cluster * (q.groups + 1));
    rank = q.cluster > 1 ? cluster_ctarank() : 0;
    const unsigned unit = blockIdx.x / q.cluster;
    tile = unit % q.tiles;
    n = unit / q.tiles;
    tx = threadIdx.x % q.tx;
    ty = threadIdx.x / q.tx;
    c = tile * q.width + tx * V;
    here = ty < q.ty && c < p.C;
    s0 = static_cast<long long>(rank) * q.rows;
    const long long left = p.S - s0;
    rows = left < 0 ? 0 : left < q.rows ? static_cast<int>(left) : q.rows;
    for (int r = threadIdx.x; r < rows; r += kThreads) valid[r] = !p.mask || p.mask[n * p.S + s0 + r];
    __syncthreads();
  }
  __device__ __forceinline__ void copy(int tensor, const Rows& r) {
    if (!here) return;
    const T* from = at<T>(r, n, s0 + ty, c);
    for (int row = ty; row < rows; row += q.ty, from += q.ty * r.row)
      if (valid[row]) copy16(smem_u32(data + (tensor * q.rows + row) * q.tx + tx), from);
  }
  __device__ __forceinline__ void get(int tensor, int row, float (&f)[V]) const {
    const uint4 u = data[(tensor * q.rows + row) * q.tx + tx];
    Vec<T, V> v;
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    unpack(v, f);
  }
  // Sums `mine` over the threads of every group and the cluster's blocks, in that order; every thread
  // gets its group's. extra: summed over blocks alone. `turn` takes the slots' halves in turn.
  __device__ __forceinline__ float2 group_sum(float2 mine, float extra, int turn, int cg, float& extra_sum) {
    red[threadIdx.x] = here ? mine : make_float2(0.f, 0.f);
    __syncthreads();
    const int stride = q.groups + 1, wide = cg / V;
    float2* half = slots + turn * q.cluster * stride;
    for (int g = warp_id(); g < q.groups; g += kThreads / 32) {
      float2 s = make_float2(0.f, 0.f);
      for (int i = lane_id(); i < wide * q.ty; i += 32) {
        const float2 v = red[i / wide * q.tx + g * wide + i % wide];
        s.x += v.x;
        s.y += v.y;
      }
      s.x = team_sum(s.x, 32);
      s.y = team_sum(s.y, 32);
      put_slot(half + rank * stride + g, s);
    }
    if (warp_id() == 0) put_slot(half + rank * stride + q.groups, make_float2(extra, 0.f));
    if (q.cluster > 1) cluster_sync();
    else __syncthreads();
    const int g = min(tx * V / cg, q.groups - 1);
    float2 s = make_float2(0.f, 0.f);
    extra_sum = 0.f;
    for (int r = 0; r < q.cluster; ++r) {
      const float2 v = half[r * stride + g];
      s.x += v.x;
      s.y += v.y;
      extra_sum += half[r * stride + q.groups].x;
    }
    return s;
  }
  // lane r writes v to block r's copy
  __device__ __forceinline__ void put_slot(float2* slot, float2 v) {
    const int r = lane_id();
    if (r >= q.cluster) return;
    if (q.cluster == 1) {
      *slot = v;
    } else {
      const uint32_t to = mapa_shared(smem_u32(slot), r);
      st_cluster_u32(to, __float_as_uint(v.x));
      st_cluster_u32(to + 4, __float_as_uint(v.y));
    }
  }
  __device__ __forceinline__ float valid_rows() const {  // of this block, in every thread of warp 0
    int k = 0;
    for (int r = lane_id(); r < rows; r += 32) k += valid[r];
#pragma unroll
    for (int o = 16; o; o >>= 1) k += __shfl_xor_sync(~0u, k, o);
    return static_cast<float>(k);
  }
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 4) norm_hold_forward_kernel(const NormParams p, const HoldPlan q) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  Hold<T, V, 1> h(p, q, dynamic);
  const int cg = p.C / p.G;
  h.copy(0, p.x);
  copies_commit();
  float w[V], b[V];
  weights<V>(p.w, h.c, h.here, 1.f, w);
  weights<V>(p.b, h.c, h.here, 0.f, b);
  if (q.cluster > 1) cluster_sync();  // every block runs before another writes to it
  copies_wait<0>();
  float sum = 0.f, count;
  if (h.here)
    for (int row = h.ty; row < h.rows; row += q.ty)
      if (h.valid[row]) {
        float f[V];
        h.get(0, row, f);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += f[e];
      }
  const float2 total = h.group_sum(make_float2(sum, 0.f), h.valid_rows(), 0, cg, count);
  const float share = 1.f / fmaxf(count * cg, 1.f);
  float mean = p.center ? total.x * share : 0.f;
  const uint64_t minus = f2_pack(-mean, -mean);
  uint64_t off = 0, squares = 0;
  if (h.here)
    for (int row = h.ty; row < h.rows; row += q.ty)
      if (h.valid[row]) {
        float f[V];
        h.get(0, row, f);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const uint64_t d = f2_add(f2_pack(f[e], f[e + 1]), minus);
          off = f2_add(off, d);
          squares = f2_fma(d, d, squares);
        }
      }
  // the sum of up to 400 values a thread left the mean off by a few of its steps, which the differences show
  const float2 o = f2_unpack(off), sq = f2_unpack(squares);
  float2 about = h.group_sum(make_float2(o.x + o.y, sq.x + sq.y), 0.f, 1, cg, count);
  about.x = p.center ? about.x * share : 0.f;
  mean += about.x;
  float var = fmaf(-about.x, about.x, about.y * share);
  if (var < 0.f) var = 0.f;  // and not fmaxf(), which would make 0 of a NaN
  const float rstd = 1.f / sqrtf(var + p.eps);
  if (!h.here) return;
  if (p.stats && h.rank == 0 && h.ty == 0 && h.c % cg == 0)
    *reinterpret_cast<float2*>(p.stats + 2 * (h.n * p.G + h.c / cg)) = make_float2(mean, rstd);
#pragma unroll
  for (int e = 0; e < V; ++e) w[e] *= rstd;
  by_act(p.act, p.gate.ptr, [&](auto kind, auto gated) {
    T* to = at<T>(p.y, h.n, h.s0 + h.ty, h.c);
    const T* gp = at<T>(p.gate, h.n, h.s0 + h.ty, h.c);
#pragma unroll 2
    for (int row = h.ty; row < h.rows; row += q.ty, to += q.ty * p.y.row, gp += q.ty * p.gate.row) {
      Vec<T, V> y = zeros<T, V>();
      if (h.valid[row]) {
        float f[V], g[V];
        if (gated) unpack(load<T, V>(gp), g);
        h.get(0, row, f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = fmaf(f[e] - mean, w[e], b[e]);
          f[e] = gated ? v * act<kind>(g[e]) : act<kind>(v);
        }
        y = pack<T, V>(f);
      }
      store<T, V>(to, y);
    }
  });
}

// Weight gradients: partial sums of every block as chan[(n * cluster + rank)][2][C].
template <typename T, int V, bool GATED>
__global__ void __launch_bounds__(kThreads, GATED ? 2 : 3) norm_hold_backward_kernel(const NormParams p, const HoldPlan q, float* chan) {
  griddep_launch();
  extern __shared__ __align__(16) uint8_t dynamic[];
  Hold<T, V, GATED ? 3 : 2> h(p, q, dynamic);
  const int cg = p.C / p.G;
  h.copy(0, p.x);
  h.copy(1, p.dy);
  if (GATED) h.copy(2, p.gate);
  copies_commit();
  float w[V], b[V], dw[V] = {}, db[V] = {};
  weights<V>(p.w, h.c, h.here, 1.f, w);
  weights<V>(p.b, h.c, h.here, 0.f, b);
  const float2 st = h.here ? *reinterpret_cast<const float2*>(p.stats + 2 * (h.n * p.G + h.c / cg)) : make_float2(0.f, 0.f);
  if (q.cluster > 1) cluster_sync();
  copies_wait<0>();
  float2 sums = make_float2(0.f, 0.f);
  by_act(p.act, GATED, [&](auto kind, auto) {
    if (h.here)
      for (int row = h.ty; row < h.rows; row += q.ty)
        if (h.valid[row]) {
          float x[V], dy[V], g[V], dg;
          h.get(0, row, x);
          h.get(1, row, dy);
          if (GATED) h.get(2, row, g);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float xh = (x[e] - st.x) * st.y;
            const float t = grad_v<kind, GATED>(fmaf(xh, w[e], b[e]), dy[e], GATED ? g[e] : 0.f, dg);
            dw[e] = fmaf(t, xh, dw[e]);
            db[e] += t;
          }
        }
  });
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sums.x = fmaf(db[e], w[e], sums.x);
    sums.y = fmaf(dw[e], w[e], sums.y);
  }
  float count;
  sums = h.group_sum(sums, h.valid_rows(), 0, cg, count);
  const float elements = fmaxf(count * cg, 1.f), m1 = p.center ? sums.x / elements : 0.f, m2 = sums.y / elements;
  by_act(p.act, GATED, [&](auto kind, auto) {
    if (!h.here) return;
    T* ox = at<T>(p.dx, h.n, h.s0 + h.ty, h.c);
    T* og = at<T>(p.dgate, h.n, h.s0 + h.ty, h.c);
    for (int row = h.ty; row < h.rows; row += q.ty, ox += q.ty * p.dx.row, og += q.ty * p.dgate.row) {
      Vec<T, V> dx = zeros<T, V>(), dgate = dx;
      if (h.valid[row]) {
        float x[V], dy[V], g[V], dg[V];
        h.get(0, row, x);
        h.get(1, row, dy);
        if (GATED) h.get(2, row, g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (x[e] - st.x) * st.y;
          const float t = grad_v<kind, GATED>(fmaf(xh, w[e], b[e]), dy[e], GATED ? g[e] : 0.f, dg[e]) * w[e];
          x[e] = (t - m1 - xh * m2) * st.y;
        }
        dx = pack<T, V>(x);
        if (GATED) dgate = pack<T, V>(dg);
      }
      store<T, V>(ox, dx);
      if (GATED) store<T, V>(og, dgate);
    }
  });
  if (!p.dw && !p.db) return;
  // the block's sum of every channel, its rows in order, through the place of x
  __syncthreads();
  float2* cell = reinterpret_cast<float2*>(dynamic);
  if (h.here)
#pragma unroll
    for (int e = 0; e < V; ++e) cell[h.ty * q.width + h.tx * V + e] = make_float2(dw[e], db[e]);
  __syncthreads();
  float* out = chan + (h.n * q.cluster + h.rank) * 2 * p.C;
  for (int i = threadIdx.x; i < q.width && h.tile * q.width + i < p.C; i += kThreads) {
    float2 s = cell[i];
    for (int r = 1; r < q.ty; ++r) {
      s.x += cell[r * q.width + i].x;
      s.y += cell[r * q.width + i].y;
    }
    out[h.tile * q.width + i] = s.x;
    out[p.C + h.tile * q.width + i] = s.y;
  }
}

// ---------------------------------------------------------------- plans and launches
bool aligned16(const Rows& r, int dtype) {
  const int run = dtype == kF32 ? 4 : 8;
  return !r.ptr || (reinterpret_cast<uintptr_t>(r.ptr) % 16 == 0 && r.batch % run == 0 && r.row % run == 0);
}

// Elements an access takes: 16 bytes where every row of every tensor allows it.
int vector_of(const NormParams& p) {
  const int run = p.dtype == kF32 ? 4 : 8;
  const bool ok = p.C / p.G % run == 0 && aligned16(p.x, p.dtype) && aligned16(p.gate, p.dtype) && aligned16(p.y, p.dtype) &&
                  aligned16(p.dy, p.dtype) && aligned16(p.dx, p.dtype) && aligned16(p.dgate, p.dtype) &&
                  reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && reinterpret_cast<uintptr_t>(p.b) % 16 == 0;
  return ok ? run : 1;
}

// Values of a row a lane holds at most: 32, or 16 where they are loaded one by one.
int lane_values(int v) { return v == 1 ? 16 : 32; }
bool rows_form(const NormParams& p, int v) { return p.S == 1 && p.C / p.G <= kThreads * lane_values(v); }

RowPlan row_plan(const NormParams& p, int v, int per_sm) {
  const int vectors = (p.C / p.G + v - 1) / v;
  RowPlan q;
  q.team = 1;
  while (q.team < 32 && q.team < vectors) q.team *= 2;
  if (p.C / p.G > 32 * lane_values(v)) q.team = kThreads;
  const int teams = kThreads / q.team;
  q.gs = p.G < teams ? p.G : teams;
  q.rpi = teams / q.gs;
  q.slices = (p.G + q.gs - 1) / q.gs;
  const long long most = (p.N + q.rpi - 1) / q.rpi;
  const long long want = (static_cast<long long>(p.sms) * per_sm + q.slices - 1) / q.slices;
  q.blocks = static_cast<int>(most < want ? most : want);
  if (q.blocks > 65535) q.blocks = 65535;
  return q;
}

// Rows and channels of a block: as many rows at once as there are, up to 32, and chunks so that a
// thread sums at most 64 rows and the blocks fill the SMs' places once (a second wave that is half
// empty cost a third of the time at 8 x 2048 x 1024).
BlockPlan block_plan(const NormParams& p, int v, int per_sm) {
  BlockPlan q;
  q.ty = 1;
  while (q.ty < 32 && q.ty < p.S) q.ty *= 2;
  q.tx = kThreads / q.ty;
  while (q.tx > 1 && (q.tx / 2) * v >= p.C && q.ty < kThreads) q.tx /= 2, q.ty *= 2;
  q.width = q.tx * v;
  q.tiles = (p.C + q.width - 1) / q.width;
  const long long blocks = p.N * q.tiles, rows_at_once = (p.S + q.ty - 1) / q.ty;
  long long chunks = static_cast<long long>(per_sm) * p.sms / blocks;
  const long long least = (rows_at_once + 63) / 64, most = rows_at_once < 512 ? rows_at_once : 512;
  if (chunks < least) chunks = least;
  if (chunks > most) chunks = most;
  q.rows = static_cast<int>((rows_at_once + chunks - 1) / chunks) * q.ty;
  q.chunks = static_cast<int>((p.S + q.rows - 1) / q.rows);
  q.segments = p.G + q.tiles;
  return q;
}

// Whether samples can be held in shared memory, and how: tiles of whole groups from 128 bytes on,
// and of 48 KB a block (three or four blocks an SM, one loading while another computes: 78 us for the
// training pass of 8 x 2048 x 1024 with padding, 88 with two of 64 KB) to the 200 KB that each
// of a cluster's eight blocks can hold at most; with few samples and tiles more blocks, down to
// two rows a thread.
bool hold_plan(const NormParams& p, int v, int tensors, HoldPlan& q) {
  const int cg = p.C / p.G, least = 8 * v;
  if (v == 1 || p.S < 2 || cg > kThreads * v) return false;
  q.width = (least + cg - 1) / cg * cg;
  if (q.width > p.C) q.width = p.C;
  q.groups = q.width / cg;
  q.tx = q.width / v;
  q.ty = kThreads / q.tx;
  if (q.ty > p.S) q.ty = static_cast<int>(p.S);
  q.tiles = (p.C + q.width - 1) / q.width;
  const long long bytes = p.S * q.tx * 16 * tensors, units = p.N * q.tiles;
  long long c = (bytes + 48 * 1024 - 1) / (48 * 1024);
  if (c > kMaxHold) c = kMaxHold;
  while (c < kMaxHold && units * c < 2LL * p.sms && p.S / (c + 1) >= 2 * q.ty) ++c;
  const long long rows = (p.S + c - 1) / c;
  if (rows * q.tx * 16 * tensors > 200 * 1024 || units * c > 0x7fffffffLL) return false;
  q.rows = static_cast<int>(rows);
  q.cluster = static_cast<int>(c);
  long long data = rows * q.tx * 16 * tensors;
  const long long cells = static_cast<long long>(q.ty) * q.width * 8;
  if (tensors > 1 && data < cells) return false;  // the weights' sums take the place of x in the end
  // with one or two vectors a row the rows' valid marks alone pass what 200 KB of rows leave
  const long long shared = data + kThreads * 8 + 2 * c * (q.groups + 1) * 8 + rows;
  if (shared > kHoldShared) return false;
  q.shared = static_cast<int>(shared);
  return true;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the block form: segments, valid rows, and with gradients the channels' sums.
struct BlockSpace {
  float2* seg;
  float *rows_of, *chan;
  size_t bytes;
  BlockSpace(const NormParams& p, const BlockPlan& q, bool backward) {
    const size_t parts = static_cast<size_t>(p.N) * q.chunks;
    uint8_t* at = static_cast<uint8_t*>(p.workspace);
    seg = reinterpret_cast<float2*>(at);
    const size_t a = round256(parts * q.segments * 8), b = round256(parts * 4);
    rows_of = reinterpret_cast<float*>(at + a);
    chan = reinterpret_cast<float*>(at + a + b);
    bytes = a + b + (backward ? round256(parts * p.C * 8) : 0);
  }
};

template <typename F>
void by_type(int dtype, int v, F&& f) {
  auto by_vec = [&](auto t) {
    if (v == 1) f(t, std::integral_constant<int, 1>{});
    else f(t, std::integral_constant<int, 16 / sizeof(t)>{});
  };
  if (dtype == kBF16) by_vec(__nv_bfloat16{});
  else if (dtype == kF16) by_vec(__half{});
  else by_vec(float{});
}
// f(vectors a lane, TEAM) for the smallest number that holds a group
template <int V, typename F>
void by_vectors(const NormParams& p, const RowPlan& q, F&& f) {
  const int need = (p.C / p.G + q.team * V - 1) / (q.team * V);
  auto with = [&](auto nv) {
    if (q.team > 32) f(nv, std::integral_constant<int, kThreads>{});
    else f(nv, std::integral_constant<int, 32>{});
  };
  if (q.team < 32) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 0>{});
  else if (need <= 1) with(std::integral_constant<int, 1>{});
  else if (need <= 2) with(std::integral_constant<int, 2>{});
  else if (need <= 4) with(std::integral_constant<int, 4>{});
  else if constexpr (V <= 4) {
    if (need <= 8) with(std::integral_constant<int, 8>{});
    else if constexpr (V == 1) with(std::integral_constant<int, 16>{});
  }
}

constexpr int kRowBlocks = 3, kRowBlocksBackward = 2;  // blocks an SM of the rows form
constexpr int kBlocks = 3, kBlocksBackward = 2;         // and of the block form

// Launches a kernel that may start while its predecessor drains: it waits (griddep_wait) before it
// reads what that one wrote.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, int shared, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

template <auto kernel, typename... Args>
cudaError_t launch_hold(const HoldPlan& q, const NormParams& p, cudaStream_t st, const Args&... args) {
  cudaError_t e = allow_shared<kernel>(kHoldShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.N * q.tiles * q.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = q.shared;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = q.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_weights(const NormParams& p, const float* part, int rows, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.dw || p.db) e = launch_after(norm_weights_kernel, dim3((p.C + 31) / 32), dim3(32, 32), 0, st, p, part, rows);
  return e;
}

}  // namespace

// The workspace must not depend on alignment, which the size query does not know: the larger of both forms.
size_t norm_workspace(const NormParams& p, bool backward) {
  size_t most = 0;
  for (int v : {1, p.dtype == kF32 ? 4 : 8}) {
    if (v > 1 && p.C / p.G % v) continue;
    size_t n;
    if (rows_form(p, v)) {
      n = backward ? static_cast<size_t>(row_plan(p, v, kRowBlocksBackward).blocks) * 2 * p.C * 4 : 0;
    } else {
      n = BlockSpace(p, block_plan(p, v, backward ? kBlocksBackward : kBlocks), backward).bytes;
      HoldPlan q;
      for (int tensors : {2, 3})
        if (backward && hold_plan(p, v, tensors, q)) {
          const size_t m = static_cast<size_t>(p.N) * q.cluster * 2 * p.C * 4;
          n = m > n ? m : n;
        }
    }
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_norm_forward(const NormParams& p, cudaStream_t st) {
  const int v = vector_of(p);
  cudaError_t e = cudaSuccess;
  by_type(p.dtype, v, [&](auto t, auto vec) {
    using T = decltype(t);
    constexpr int V = decltype(vec)::value;
    if (rows_form(p, v)) {
      const RowPlan q = row_plan(p, v, kRowBlocks);
      by_vectors<V>(p, q, [&](auto nv, auto team) {
        e = launch_plain(norm_rows_forward_kernel<T, V, decltype(nv)::value, decltype(team)::value>, dim3(q.slices, q.blocks),
                         dim3(kThreads), 0, st, p, q);
      });
    } else if (HoldPlan hold; hold_plan(p, v, 1, hold)) {
      if constexpr (V > 1) e = launch_hold<norm_hold_forward_kernel<T, V>>(hold, p, st, p, hold);
    } else {
      const BlockPlan q = block_plan(p, v, kBlocks);
      const BlockSpace s(p, q, false);
      const long long grid = p.N * q.chunks * q.tiles;
      if (grid > 0x7fffffffLL) {
        e = cudaErrorInvalidConfiguration;
        return;
      }
      e = launch_plain(norm_sums_kernel<T, V>, dim3(unsigned(grid)), dim3(kThreads), 0, st, p, q, s.seg, s.rows_of);
      if (e != cudaSuccess) return;
      e = launch_after(norm_apply_kernel<T, V>, dim3(unsigned(grid)), dim3(kThreads), (q.width + 1) * 8, st, p, q,
                       static_cast<const float2*>(s.seg), static_cast<const float*>(s.rows_of));
    }
  });
  return e;
}

cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t st) {
  const int v = vector_of(p);
  cudaError_t e = cudaSuccess;
  by_type(p.dtype, v, [&](auto t, auto vec) {
    using T = decltype(t);
    constexpr int V = decltype(vec)::value;
    if (rows_form(p, v)) {
      const RowPlan q = row_plan(p, v, kRowBlocksBackward);
      const int sums = (q.rpi - 1) * q.gs * (p.C / p.G) * 8;
      by_vectors<V>(p, q, [&](auto nv, auto team) {
        constexpr auto kernel = norm_rows_backward_kernel<T, V, decltype(nv)::value, decltype(team)::value>;
        // a block's sums need at most 8 bytes for each of its threads' values
        constexpr int kRows = kAhead * kRowStage<T, V, decltype(nv)::value>, kSums = kThreads * V * decltype(nv)::value * 8;
        constexpr int kShared = kRows > kSums ? kRows : kSums;
        e = allow_shared<kernel>(kShared);
        if (e == cudaSuccess)
          e = launch_plain(kernel, dim3(q.slices, q.blocks), dim3(kThreads), kRows > sums ? kRows : sums, st, p, q);
      });
      if (e == cudaSuccess) e = launch_weights(p, static_cast<const float*>(p.workspace), q.blocks, st);
    } else if (HoldPlan hold; hold_plan(p, v, p.gate.ptr ? 3 : 2, hold)) {
      if constexpr (V > 1) {
        float* chan = static_cast<float*>(p.workspace);
        e = p.gate.ptr ? launch_hold<norm_hold_backward_kernel<T, V, true>>(hold, p, st, p, hold, chan)
                       : launch_hold<norm_hold_backward_kernel<T, V, false>>(hold, p, st, p, hold, chan);
        if (e == cudaSuccess) e = launch_weights(p, chan, static_cast<int>(p.N * hold.cluster), st);
      }
    } else {
      const BlockPlan q = block_plan(p, v, kBlocksBackward);
      const BlockSpace s(p, q, true);
      const long long grid = p.N * q.chunks * q.tiles, parts = p.N * q.chunks;
      if (grid > 0x7fffffffLL) {
        e = cudaErrorInvalidConfiguration;
        return;
      }
      e = launch_plain(norm_grad_sums_kernel<T, V>, dim3(unsigned(grid)), dim3(kThreads), kThreads * V * 8, st, p, q, s.chan,
                       s.seg, s.rows_of);
      if (e != cudaSuccess) return;
      e = launch_after(norm_grad_apply_kernel<T, V>, dim3(unsigned(grid)), dim3(kThreads), (q.width + 1) * 8, st, p, q,
                       static_cast<const float2*>(s.seg), static_cast<const float*>(s.rows_of));
      if (e == cudaSuccess) e = launch_weights(p, s.chan, static_cast<int>(parts), st);
    }
  });
  return e;
}

}  // namespace msgla
