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
// A padded row has c = 0 and u = 0 and is not read: its logit is taken as +inf.
//
// Bound: HBM. Forward 3 tensors a pass (x, z in, h out), backward 5 (x, z, dh in, dx, dz
// out); the forward states that the backward needs are rebuilt from one saved f32
// state per 64 rows (3 % of a 16-bit tensor), which costs less than reading h would and
// keeps them in 32 bits. The next bound is the issue rate: at the full rate of HBM the
// SMs have 33 (forward) and 55 (backward) issue slots an element, so the gate runs on
// packed f32x2 polynomials with one ex2 an element.
//
// Split: channels are independent, rows are a chain. A block takes 64 channels (two a
// lane, so a warp reads whole 128-byte lines of 16-bit rows) and W x R rows at a time,
// every warp R neighbouring rows held in registers: one pass over them gives the warp's
// decay product and local end state, the W warps' are joined in shared memory, and a
// second pass over the registers gives the rows from the true start. Where one block
// per channel tile leaves SMs idle, a cluster of 2, 4 or 8 blocks shares the tile's rows
// and passes the joined pairs through distributed shared memory, one cluster barrier a
// step. The next step's rows are loaded before this step's are joined.
#include <cmath>
#include <type_traits>

#include "ops_internal.h"
#include "sm100_ptx.cuh"

namespace msgla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 64;  // channels per block
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- pairs of elements
// Two neighbouring channels of one row, as loaded.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw zero() { return 0u; }
  static __device__ __forceinline__ Raw inf() { return 0x7f807f80u; }
  static __device__ __forceinline__ uint64_t f32(Raw r) {
    return f2_pack(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  static __device__ __forceinline__ Raw round(uint64_t v) {
    const float2 f = f2_unpack(v);
    return pack_bf162(f.x, f.y);
  }
  static __device__ __forceinline__ Raw join(__nv_bfloat16 a, __nv_bfloat16 b) {
    return uint32_t(__bfloat16_as_ushort(a)) | uint32_t(__bfloat16_as_ushort(b)) << 16;
  }
  static __device__ __forceinline__ __nv_bfloat16 half(Raw r, int i) {
    return __ushort_as_bfloat16(static_cast<unsigned short>(i ? r >> 16 : r & 0xffffu));
  }
};
template <>
struct Pair<__half> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw zero() { return 0u; }
  static __device__ __forceinline__ Raw inf() { return 0x7c007c00u; }
  static __device__ __forceinline__ uint64_t f32(Raw r) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
    return f2_pack(f.x, f.y);
  }
  static __device__ __forceinline__ Raw round(uint64_t v) {
    const float2 f = f2_unpack(v);
    return pack_half2(f.x, f.y);
  }
  static __device__ __forceinline__ Raw join(__half a, __half b) {
    return uint32_t(__half_as_ushort(a)) | uint32_t(__half_as_ushort(b)) << 16;
  }
  static __device__ __forceinline__ __half half(Raw r, int i) {
    return __ushort_as_half(static_cast<unsigned short>(i ? r >> 16 : r & 0xffffu));
  }
};
template <>
struct Pair<float> {
  using Raw = uint64_t;
  static __device__ __forceinline__ Raw zero() { return 0ull; }
  static __device__ __forceinline__ Raw inf() { return 0x7f8000007f800000ull; }
  static __device__ __forceinline__ uint64_t f32(Raw r) { return r; }
  static __device__ __forceinline__ Raw round(uint64_t v) { return v; }
  static __device__ __forceinline__ Raw join(float a, float b) { return f2_pack(a, b); }
  static __device__ __forceinline__ float half(Raw r, int i) {
    const float2 f = f2_unpack(r);
    return i ? f.y : f.x;
  }
};

// Loads and stores of a pair; PAIRED: both channels exist wherever the first does and
// the address is aligned to the pair. `n` is the number of the pair's channels inside D.
template <typename T, bool PAIRED>
__device__ __forceinline__ typename Pair<T>::Raw load_pair(const T* p, int n, typename Pair<T>::Raw none) {
  using P = Pair<T>;
  if (PAIRED) return n ? __ldg(reinterpret_cast<const typename P::Raw*>(p)) : none;
  return n ? P::join(p[0], n > 1 ? p[1] : P::half(none, 1)) : none;
}
template <typename T, bool PAIRED>
__device__ __forceinline__ void store_pair(T* p, int n, typename Pair<T>::Raw v) {
  using P = Pair<T>;
  if (PAIRED) {
    if (n) *reinterpret_cast<typename P::Raw*>(p) = v;
  } else {
    if (n) p[0] = P::half(v, 0);
    if (n > 1) p[1] = P::half(v, 1);
  }
}
// f32 states [.., D]: 8-byte accesses where the pairs are aligned (D even)
template <bool PAIRED>
__device__ __forceinline__ uint64_t load_state(const float* p, int n) {
  if (PAIRED) return n ? *reinterpret_cast<const uint64_t*>(p) : 0ull;
  return f2_pack(n ? p[0] : 0.f, n > 1 ? p[1] : 0.f);
}
template <bool PAIRED>
__device__ __forceinline__ void store_state(float* p, int n, uint64_t v) {
  if (PAIRED) {
    if (n) *reinterpret_cast<uint64_t*>(p) = v;
  } else {
    const float2 f = f2_unpack(v);
    if (n) p[0] = f.x;
    if (n > 1) p[1] = f.y;
  }
}

// ---------------------------------------------------------------- the gate
// log(1 + e) / e on [0, 1] and (e^{-s} - 1) / s on [0, 1]: Chebyshev expansions cut off
// at degree 7 and 5 (relative errors 2.2e-7 and 8e-8, computed in 64 bits).
__device__ __forceinline__ uint64_t log1p_over(uint64_t e) {
  constexpr float k[8] = {0.999999762f, -0.499971271f, 0.332711875f, -0.244704694f, 0.176754937f, -0.106677905f, 0.0433708504f, -0.00833649747f};
  uint64_t r = f2_both(k[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) r = f2_fma(r, e, f2_both(k[i]));
  return r;
}
__device__ __forceinline__ uint64_t expm1_over(uint64_t s) {
  constexpr float k[6] = {-0.99999994f, 0.499994457f, -0.16660437f, 0.0414042994f, -0.00782115851f, 0.000906161731f};
  uint64_t r = f2_both(k[5]);
#pragma unroll
  for (int i = 4; i >= 0; --i) r = f2_fma(r, s, f2_both(k[i]));
  return r;
}

// -c of two logits, and with DOWN also a (1 - sigmoid(z)) / tau. For f32 tensors the
// library functions: their callers compare 24 bits, and 12 bytes an element leave time.
// TAU1: c = 1 - sigmoid(z) in closed form, one ex2 and one reciprocal.
template <typename T, bool TAU1, bool DOWN>
__device__ __forceinline__ uint64_t neg_decay(uint64_t z, float inv_tau, uint64_t& down) {
  const float2 f = f2_unpack(z);
  if constexpr (sizeof(T) == 4) {
    float nc[2], d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float v = i ? f.y : f.x, e = expf(-fabsf(v));
      const float dn = (v >= 0.f ? e : 1.f) / (1.f + e);
      nc[i] = TAU1 ? -dn : expm1f(-(log1pf(e) + fmaxf(-v, 0.f)) * inv_tau);
      if (DOWN) d[i] = dn * (1.f + nc[i]) * inv_tau;
    }
    if (DOWN) down = f2_pack(d[0], d[1]);
    return f2_pack(nc[0], nc[1]);
  } else {
    const float e0 = ex2_approx(-kLog2e * fabsf(f.x)), e1 = ex2_approx(-kLog2e * fabsf(f.y));
    float d0, d1;
    if (TAU1 || DOWN) {
      d0 = (f.x >= 0.f ? e0 : 1.f) * rcp_approx(1.f + e0);
      d1 = (f.y >= 0.f ? e1 : 1.f) * rcp_approx(1.f + e1);
    }
    uint64_t nc;
    if (TAU1) {
      nc = f2_pack(-d0, -d1);
    } else {
      const uint64_t e = f2_pack(e0, e1);
      uint64_t s = f2_fma(e, log1p_over(e), f2_pack(fmaxf(-f.x, 0.f), fmaxf(-f.y, 0.f)));
      s = f2_mul(s, f2_both(inv_tau));
      nc = f2_mul(s, expm1_over(s));
      const float2 sf = f2_unpack(s);
      if (fmaxf(sf.x, sf.y) > 1.f) {  // outside the expansion's interval; e^{-s} < 0.37 loses nothing in the difference
        float2 n = f2_unpack(nc);
        if (sf.x > 1.f) n.x = ex2_approx(-kLog2e * sf.x) - 1.f;
        if (sf.y > 1.f) n.y = ex2_approx(-kLog2e * sf.y) - 1.f;
        nc = f2_pack(n.x, n.y);
      }
    }
    if (DOWN) down = f2_mul(f2_mul(f2_pack(d0, d1), f2_both(inv_tau)), f2_add(nc, f2_both(1.f)));
    return nc;
  }
}

// h - c h + u
__device__ __forceinline__ uint64_t advance(uint64_t h, uint64_t nc, uint64_t x, bool tied) {
  h = f2_fma(nc, h, h);
  return tied ? f2_fma(nc, f2_neg(x), h) : f2_add(h, x);
}

// ---------------------------------------------------------------- blocks and clusters
// What W warps hand over: the decay product and local end value of their rows.
struct alignas(16) Join {
  uint64_t p, v;
};

// Sends this block's pair to every block of the cluster and waits for all of them.
__device__ __forceinline__ void send_join(Join* slots, int rank, int cluster, const Join& j, bool sender) {
  if (sender) {
    const uint32_t at = smem_u32(slots + rank * 32 + lane_id());
    for (int r = 0; r < cluster; ++r)
      asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(mapa_shared(at, r)), "l"(j.p), "l"(j.v) : "memory");
  }
  cluster_sync();
}

// Bits of the valid rows t0 .. t0 + R - 1 (bit r: row t0 + r).
template <int R>
__device__ __forceinline__ uint32_t valid_rows(const uint8_t* m, int t0, int L) {
  const int n = min(max(L - t0, 0), R);
  if (!m) return (1u << n) - 1u;
  const int r = lane_id();
  return __ballot_sync(~0u, r < n && m[t0 + r] != 0);
}

// ---------------------------------------------------------------- forward
template <typename T, int W, int R, bool PAIRED, bool TAU1>
__global__ void __launch_bounds__(W * 32, W == 8 ? 2 : 1) scan_forward_kernel(const ScanParams p) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int kRows = W * R;
  static_assert(R <= 32 && kScanSave % R == 0, "saved states start a warp's rows");
  __shared__ Join warps[W][32];
  __shared__ Join blocks[2][kMaxCluster * 32];
  const int cluster = p.cluster, rank = cluster > 1 ? cluster_ctarank() : 0;
  const int w = warp_id(), lane = lane_id(), b = blockIdx.y;
  const int ch = blockIdx.x / cluster * kTile + 2 * lane, n = min(max(p.D - ch, 0), 2);
  const bool tied = p.tied;
  const T* x = static_cast<const T*>(p.x.ptr) + b * p.x.batch + ch;
  const T* z = static_cast<const T*>(p.z.ptr) + b * p.z.batch + ch;
  T* o = static_cast<T*>(p.h.ptr) + b * p.h.batch + ch;
  const uint8_t* m = p.mask ? p.mask + static_cast<size_t>(b) * p.L : nullptr;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  const int nsave = (p.L + kScanSave - 1) / kScanSave;
  const int steps = (p.L + cluster * kRows - 1) / (cluster * kRows);

  Raw xr[R], zr[R];
  uint32_t bits;
  auto load = [&](int t0) {
    bits = valid_rows<R>(m, t0, p.L);
    const T* xp = x + static_cast<long long>(t0) * p.x.row;
    const T* zp = z + static_cast<long long>(t0) * p.z.row;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int k = bits >> r & 1 ? n : 0;
      xr[r] = load_pair<T, PAIRED>(xp + r * p.x.row, k, P::zero());
      zr[r] = load_pair<T, PAIRED>(zp + r * p.z.row, k, P::inf());
    }
  };

  uint64_t carry = p.h0 ? load_state<PAIRED>(p.h0 + state_at, n) : 0ull;
  load((rank * W + w) * R);
  if (cluster > 1) cluster_sync();  // every block runs before another writes to it
  for (int step = 0; step < steps; ++step) {
    const int t0 = ((step * cluster + rank) * W + w) * R;
    uint64_t nc[R], unused, prod = f2_both(1.f), h = 0ull;
    Raw xs[R];
    const uint32_t now = bits;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      xs[r] = xr[r];
      nc[r] = neg_decay<T, TAU1, false>(P::f32(zr[r]), p.inv_tau, unused);
    }
    if (step + 1 < steps) load(t0 + cluster * kRows);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h = advance(h, nc[r], P::f32(xs[r]), tied);
      prod = f2_fma(nc[r], prod, prod);
    }
    warps[w][lane] = Join{prod, h};
    __syncthreads();
    Join before{f2_both(1.f), 0ull}, all{f2_both(1.f), 0ull};
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (j == w) before = all;
      const Join q = warps[j][lane];
      all.v = f2_fma(q.p, all.v, q.v);
      all.p = f2_mul(q.p, all.p);
    }
    uint64_t start = carry;
    if (cluster > 1) {
      Join* slots = blocks[step & 1];
      send_join(slots, rank, cluster, all, w == 0);
      for (int j = 0; j < cluster; ++j) {
        if (j == rank) start = carry;
        const Join q = slots[j * 32 + lane];
        carry = f2_fma(q.p, carry, q.v);
      }
    } else {
      carry = f2_fma(all.p, carry, all.v);
      __syncthreads();  // the next step writes `warps`
    }
    h = f2_fma(before.p, start, before.v);
    if (p.saved && t0 % kScanSave == 0 && t0 < p.L)
      store_state<PAIRED>(p.saved + (static_cast<size_t>(b) * nsave + t0 / kScanSave) * p.D + ch, n, h);
    T* op = o + static_cast<long long>(t0) * p.h.row;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h = advance(h, nc[r], P::f32(xs[r]), tied);
      if (t0 + r < p.L) store_pair<T, PAIRED>(op + r * p.h.row, n, now >> r & 1 ? P::round(h) : P::zero());
    }
  }
  if (rank == 0 && w == 0) store_state<PAIRED>(p.last + state_at, n, carry);
}

// ---------------------------------------------------------------- backward
// Blocks of 64 rows, from the last: rank 0 of a cluster takes the latest. A warp's rows
// hand a_t g_t of their first row down to the rows before: in = P out + G.
template <typename T, int W, int R, bool PAIRED, bool TAU1>
__global__ void __launch_bounds__(W * 32, W == 8 ? 2 : 1) scan_backward_kernel(const ScanParams p) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  static_assert(W * R == kScanSave, "a block's rows start from a saved state");
  __shared__ Join warps[W][32];
  __shared__ uint64_t grads[W][32];
  __shared__ Join blocks[2][kMaxCluster * 32];
  const int cluster = p.cluster, rank = cluster > 1 ? cluster_ctarank() : 0;
  const int w = warp_id(), lane = lane_id(), b = blockIdx.y;
  const int ch = blockIdx.x / cluster * kTile + 2 * lane, n = min(max(p.D - ch, 0), 2);
  const bool tied = p.tied;
  const T* x = static_cast<const T*>(p.x.ptr) + b * p.x.batch + ch;
  const T* z = static_cast<const T*>(p.z.ptr) + b * p.z.batch + ch;
  const T* d = static_cast<const T*>(p.dh.ptr) + (p.dh.ptr ? b * p.dh.batch + ch : 0);
  const bool has_d = p.dh.ptr != nullptr;
  T* ox = static_cast<T*>(p.dx.ptr) + b * p.dx.batch + ch;
  T* oz = static_cast<T*>(p.dz.ptr) + b * p.dz.batch + ch;
  const uint8_t* m = p.mask ? p.mask + static_cast<size_t>(b) * p.L : nullptr;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  const int nsave = (p.L + kScanSave - 1) / kScanSave;
  const int steps = (nsave + cluster - 1) / cluster;

  Raw xr[R], zr[R], dr[R];
  uint64_t sr;
  uint32_t bits;
  auto load = [&](int k) {  // block of rows k, or none when k < 0
    const int t0 = k * kScanSave + w * R;
    bits = k < 0 ? 0u : valid_rows<R>(m, t0, p.L);
    sr = k < 0 ? 0ull : load_state<PAIRED>(p.saved + (static_cast<size_t>(b) * nsave + k) * p.D + ch, n);
    const T* xp = x + static_cast<long long>(t0) * p.x.row;
    const T* zp = z + static_cast<long long>(t0) * p.z.row;
    const T* dp = d + static_cast<long long>(t0) * p.dh.row;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int q = bits >> r & 1 ? n : 0;
      xr[r] = load_pair<T, PAIRED>(xp + r * p.x.row, q, P::zero());
      zr[r] = load_pair<T, PAIRED>(zp + r * p.z.row, q, P::inf());
      dr[r] = load_pair<T, PAIRED>(dp + r * p.dh.row, has_d ? q : 0, P::zero());
    }
  };

  uint64_t carry = p.dlast ? load_state<PAIRED>(p.dlast + state_at, n) : 0ull;
  load(nsave - 1 - rank);
  if (cluster > 1) cluster_sync();
  for (int step = 0; step < steps; ++step) {
    const int k = nsave - 1 - step * cluster - rank, t0 = k * kScanSave + w * R;
    uint64_t nc[R], slope[R], before[R], prod = f2_both(1.f), h = 0ull, g = 0ull;
    Raw xs[R], ds[R];
    const uint32_t now = bits;
    uint64_t state = sr;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      xs[r] = xr[r];
      ds[r] = dr[r];
      nc[r] = neg_decay<T, TAU1, true>(P::f32(zr[r]), p.inv_tau, slope[r]);
    }
    if (step + 1 < steps) load(k - cluster);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h = advance(h, nc[r], P::f32(xs[r]), tied);
      prod = f2_fma(nc[r], prod, prod);
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      g = f2_add(g, P::f32(ds[r]));
      g = f2_fma(nc[r], g, g);
    }
    warps[w][lane] = Join{prod, h};
    grads[w][lane] = g;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const Join q = warps[j][lane];
      if (j < w) state = f2_fma(q.p, state, q.v);
    }
    Join after{f2_both(1.f), 0ull}, all{f2_both(1.f), 0ull};
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
      if (j == w) after = all;
      const uint64_t q = warps[j][lane].p;
      all.v = f2_fma(q, all.v, grads[j][lane]);
      all.p = f2_mul(q, all.p);
    }
    uint64_t in = carry;
    if (cluster > 1) {
      Join* slots = blocks[step & 1];
      send_join(slots, rank, cluster, all, w == 0);
      for (int j = 0; j < cluster; ++j) {
        if (j == rank) in = carry;
        const Join q = slots[j * 32 + lane];
        carry = f2_fma(q.p, carry, q.v);
      }
    } else {
      carry = f2_fma(all.p, carry, all.v);
      __syncthreads();
    }
    in = f2_fma(after.p, in, after.v);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t xv = P::f32(xs[r]);
      before[r] = tied ? f2_add(state, f2_neg(xv)) : state;
      state = advance(state, nc[r], xv, tied);
    }
    T* xp = ox + static_cast<long long>(t0) * p.dx.row;
    T* zp = oz + static_cast<long long>(t0) * p.dz.row;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      g = f2_add(in, P::f32(ds[r]));
      const uint64_t gz = f2_mul(f2_mul(g, before[r]), slope[r]), gx = tied ? f2_neg(f2_mul(nc[r], g)) : g;
      in = f2_fma(nc[r], g, g);
      if (now >> r & 1) {
        store_pair<T, PAIRED>(xp + r * p.dx.row, n, P::round(gx));
        store_pair<T, PAIRED>(zp + r * p.dz.row, n, P::round(gz));
      } else {
        in = g;  // a padded row hands on what it got
        if (k >= 0 && t0 + r < p.L) {
          store_pair<T, PAIRED>(xp + r * p.dx.row, n, P::zero());
          store_pair<T, PAIRED>(zp + r * p.dz.row, n, P::zero());
        }
      }
    }
  }
  if (p.dh0 && rank == 0 && w == 0) store_state<PAIRED>(p.dh0 + state_at, n, carry);
}

// ---------------------------------------------------------------- single tokens
template <typename T, bool PAIRED, bool TAU1>
__global__ void __launch_bounds__(128) scan_step_kernel(const StepParams p) {
  using P = Pair<T>;
  const int ch = (blockIdx.x * 128 + threadIdx.x) * 2, n = min(max(p.D - ch, 0), 2), b = blockIdx.y;
  if (n == 0) return;
  typename P::Raw out = P::zero();
  if (!p.mask || p.mask[b]) {
    float* s = p.state + static_cast<size_t>(b) * p.D + ch;
    uint64_t unused;
    const uint64_t z = P::f32(load_pair<T, PAIRED>(static_cast<const T*>(p.z) + b * p.z_row + ch, n, P::inf()));
    const uint64_t x = P::f32(load_pair<T, PAIRED>(static_cast<const T*>(p.x) + b * p.x_row + ch, n, P::zero()));
    const uint64_t h = advance(load_state<PAIRED>(s, n), neg_decay<T, TAU1, false>(z, p.inv_tau, unused), x, p.tied);
    store_state<PAIRED>(s, n, h);
    out = P::round(h);
  }
  store_pair<T, PAIRED>(static_cast<T*>(p.h) + b * p.h_row + ch, n, out);
}

// ---------------------------------------------------------------- launches
// f(element type, PAIRED, TAU1) with the values as compile-time constants
template <typename F>
void by_kind(int dtype, bool paired, bool tau1, F&& f) {
  auto by_tau = [&](auto t, auto pr) {
    if (tau1) f(t, pr, std::true_type{});
    else f(t, pr, std::false_type{});
  };
  auto by_pair = [&](auto t) {
    if (paired) by_tau(t, std::true_type{});
    else by_tau(t, std::false_type{});
  };
  if (dtype == kBF16) by_pair(__nv_bfloat16{});
  else if (dtype == kF16) by_pair(__half{});
  else by_pair(float{});
}

// Whether pairs of channels are aligned in every row of r.
bool paired_rows(const Rows& r, int dtype) {
  const uintptr_t pair = dtype == kF32 ? 8 : 4;
  return !r.ptr || (reinterpret_cast<uintptr_t>(r.ptr) % pair == 0 && r.batch % 2 == 0 && r.row % 2 == 0);
}
bool paired_state(const float* s) { return reinterpret_cast<uintptr_t>(s) % 8 == 0; }

int multiprocessors() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// Blocks per channel tile: the smallest cluster among those that fill the GPU best (blocks
// in whole waves of `resident`), and no more blocks than the rows need.
int pick_cluster(int tiles, int L, int rows, int resident) {
  int best = 1;
  double best_fill = 0;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    if (c > 1 && static_cast<long long>(c / 2) * rows >= L) break;
    const double blocks = static_cast<double>(tiles) * c, waves = std::ceil(blocks / resident);
    const double fill = blocks / (waves * resident);
    if (fill > best_fill * 1.02) best = c, best_fill = fill;
  }
  return best;
}

template <typename K>
cudaError_t launch(K kernel, const ScanParams& p, int threads, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.D + kTile - 1) / kTile * p.cluster, p.B);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_scan_forward(const ScanParams& params, cudaStream_t st) {
  ScanParams p = params;
  const bool paired = p.D % 2 == 0 && paired_rows(p.x, p.dtype) && paired_rows(p.z, p.dtype) && paired_rows(p.h, p.dtype) &&
                      paired_state(p.h0) && paired_state(p.last) && paired_state(p.saved);
  cudaError_t e = cudaSuccess;
  by_kind(p.dtype, paired, p.inv_tau == 1.f, [&](auto t, auto pr, auto tau1) {
    using T = decltype(t);
    constexpr int W = 8, R = sizeof(T) == 4 ? 8 : 16;
    p.cluster = pick_cluster((p.D + kTile - 1) / kTile * p.B, p.L, W * R, 2 * multiprocessors());
    e = launch(scan_forward_kernel<T, W, R, decltype(pr)::value, decltype(tau1)::value>, p, W * 32, st);
  });
  return e;
}

cudaError_t launch_scan_backward(const ScanParams& params, cudaStream_t st) {
  ScanParams p = params;
  const bool paired = p.D % 2 == 0 && paired_rows(p.x, p.dtype) && paired_rows(p.z, p.dtype) && paired_rows(p.dh, p.dtype) &&
                      paired_rows(p.dx, p.dtype) && paired_rows(p.dz, p.dtype) && paired_state(p.saved) &&
                      paired_state(p.dlast) && paired_state(p.dh0);
  cudaError_t e = cudaSuccess;
  by_kind(p.dtype, paired, p.inv_tau == 1.f, [&](auto t, auto pr, auto tau1) {
    using T = decltype(t);
    constexpr int W = sizeof(T) == 4 ? 16 : 8, R = kScanSave / W;
    p.cluster = pick_cluster((p.D + kTile - 1) / kTile * p.B, p.L, W * R, (W == 8 ? 2 : 1) * multiprocessors());
    e = launch(scan_backward_kernel<T, W, R, decltype(pr)::value, decltype(tau1)::value>, p, W * 32, st);
  });
  return e;
}

cudaError_t launch_scan_step(const StepParams& p, cudaStream_t st) {
  const Rows rows[3] = {{const_cast<void*>(p.x), p.x_row, 0}, {const_cast<void*>(p.z), p.z_row, 0}, {p.h, p.h_row, 0}};
  bool paired = p.D % 2 == 0 && paired_state(p.state);
  for (const Rows& r : rows) paired = paired && paired_rows(r, p.dtype);
  const dim3 grid((p.D + 255) / 256, p.B);
  by_kind(p.dtype, paired, p.inv_tau == 1.f, [&](auto t, auto pr, auto tau1) {
    scan_step_kernel<decltype(t), decltype(pr)::value, decltype(tau1)::value><<<grid, 128, 0, st>>>(p);
  });
  return cudaGetLastError();
}

}  // namespace msgla
