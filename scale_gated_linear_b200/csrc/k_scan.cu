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
// An infinite h makes NaN of h - c h where a h stays infinite: channels that end so are computed
// again by the formula as it stands (see "values that are not finite").
//
// Bound: HBM. Forward 3 tensors a pass (x, z in, h out), backward 5 (x, z, dh in, dx, dz
// out); the forward states that the backward needs are rebuilt from one saved f32 state a chunk
// of 16 rows (8 of f32; an eighth of a tensor's bytes), which costs less than reading h would
// and keeps them in 32 bits. Next to it the issue rate: at HBM's rate the SMs have 33 (forward)
// and 55 (backward) issue slots an element, and spend 27 and 42. So the gate runs on packed
// f32x2 polynomials with one ex2 an element, accurate in c and not only in a: the hardware's
// log2 alone is off by 2^-22 of one, which is all of c for a gate near one.
//
// Split: channels are independent, rows are a chain. A block takes 64 channels (two a lane, so a
// warp reads whole lines), a warp a chunk of rows: copied to shared memory while the chunk
// before is computed; one pass for the chunk's decay product and local end value; then, once the
// value before it is known, a second pass for the rows, which leave through shared memory in
// 16-byte stores. How that value comes:
// * one block per tile and sequence: from warp to warp, a relay. The warps are at different places
//   of their chunks, so loads, gates and stores overlap, and one block keeps its SM busy: 90 %
//   of copy bandwidth where the tiles are a whole number an SM (296 tiles of 8192 rows, bf16),
//   68 % at 8 x 2048 x 2048, whose 256 tiles give 108 SMs two and 40 one;
// * few tiles: rows split over the blocks of a cluster, joined through distributed shared memory
//   every step (32 tiles of 16384 rows: 70 us against 158 of one block a tile).
// Before: one thread a channel 1310 us at 8 x 2048 x 2048; rows in registers with a block
// barrier a step 75; a warp of its own for the chain, fed by the others, 52; the relay 45.
#include <cmath>
#include <mutex>
#include <type_traits>

#include "ops_internal.h"
#include "sm100_ptx.cuh"

namespace msgla {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.4426950408889634 - static_cast<double>(kLog2e);
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A warp's R rows of 64 channels take 2 KB for every type (16 rows of 128 bytes, 8 of 256).
constexpr int kRowsBytes = 2048;
template <typename T>
constexpr int kRowsOf = kRowsBytes / (64 * sizeof(T));

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
  static __device__ __forceinline__ uint64_t minus(Raw r) { return f32(r ^ 0x80008000u); }
  static __device__ __forceinline__ Raw round(uint64_t v) {
    const float2 f = f2_unpack(v);
    return pack_bf162(f.x, f.y);
  }
  static __device__ __forceinline__ Raw least(Raw a, Raw b) {
    const __nv_bfloat162 m = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const Raw*>(&m);
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
  static __device__ __forceinline__ uint64_t minus(Raw r) { return f32(r ^ 0x80008000u); }
  static __device__ __forceinline__ Raw round(uint64_t v) {
    const float2 f = f2_unpack(v);
    return pack_half2(f.x, f.y);
  }
  static __device__ __forceinline__ Raw least(Raw a, Raw b) {
    const __half2 m = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const Raw*>(&m);
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
  static __device__ __forceinline__ uint64_t minus(Raw r) { return f2_neg(r); }
  static __device__ __forceinline__ Raw round(uint64_t v) { return v; }
  static __device__ __forceinline__ Raw least(Raw a, Raw b) {
    const float2 f = f2_unpack(a), g = f2_unpack(b);
    return f2_pack(fminf(f.x, g.x), fminf(f.y, g.y));
  }
  static __device__ __forceinline__ Raw join(float a, float b) { return f2_pack(a, b); }
  static __device__ __forceinline__ float half(Raw r, int i) {
    const float2 f = f2_unpack(r);
    return i ? f.y : f.x;
  }
};

// Loads and stores of a lane's pair; VEC: both channels exist wherever the first does and
// the address is aligned to the pair. `n`: channels of the pair inside D.
template <typename T, bool VEC>
__device__ __forceinline__ typename Pair<T>::Raw load_pair(const T* p, int n, typename Pair<T>::Raw none) {
  using P = Pair<T>;
  if (VEC) return n ? __ldg(reinterpret_cast<const typename P::Raw*>(p)) : none;
  return n ? P::join(p[0], n > 1 ? p[1] : P::half(none, 1)) : none;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_pair(T* p, int n, typename Pair<T>::Raw v) {
  using P = Pair<T>;
  if (VEC) {
    if (n) *reinterpret_cast<typename P::Raw*>(p) = v;
  } else {
    if (n) p[0] = P::half(v, 0);
    if (n > 1) p[1] = P::half(v, 1);
  }
}
// f32 states [.., D]: 8-byte accesses where the pairs are aligned (D even)
template <bool VEC>
__device__ __forceinline__ uint64_t load_state(const float* p, int n) {
  if (VEC) return n > 0 ? *reinterpret_cast<const uint64_t*>(p) : 0ull;
  return f2_pack(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f);
}
template <bool VEC>
__device__ __forceinline__ void store_state(float* p, int n, uint64_t v) {
  if (VEC) {
    if (n > 0) *reinterpret_cast<uint64_t*>(p) = v;
  } else {
    const float2 f = f2_unpack(v);
    if (n > 0) p[0] = f.x;
    if (n > 1) p[1] = f.y;
  }
}

// ---------------------------------------------------------------- the gate
// log(1 + e) / e on [0, 1]: Chebyshev expansions computed in 64 bits, cut off at degree 7 for 16-bit
// tensors (relative error 2.4e-7) and at 9 for f32 (6e-9, and roundings). Both halves of
// the packed operands stand in constant memory.
__constant__ float2 kLog1p7[8] = {
    {0.999999762f, 0.999999762f},   {-0.499971271f, -0.499971271f}, {0.332711875f, 0.332711875f},
    {-0.244704694f, -0.244704694f}, {0.176754937f, 0.176754937f},   {-0.106677905f, -0.106677905f},
    {0.0433708504f, 0.0433708504f}, {-0.00833649747f, -0.00833649747f}};
__constant__ float2 kLog1p9[10] = {
    {1.f, 1.f},                       {-0.499998897f, -0.499998897f}, {0.333296657f, 0.333296657f},
    {-0.249511674f, -0.249511674f},   {0.196610183f, 0.196610183f},   {-0.152632743f, -0.152632743f},
    {0.105329506f, 0.105329506f},     {-0.0562695265f, -0.0562695265f}, {0.0194876865f, 0.0194876865f},
    {-0.00316399941f, -0.00316399941f}};
template <typename T>
constexpr int kDegree = sizeof(T) == 4 ? 9 : 7;
template <typename T>
constexpr int kExpDegree = sizeof(T) == 4 ? 5 : 4;
__device__ __forceinline__ uint64_t f2_const(const float2& v) { return *reinterpret_cast<const uint64_t*>(&v); }
template <typename T>
__device__ __forceinline__ uint64_t log1p_term(int i) {
  if constexpr (sizeof(T) == 4) return f2_const(kLog1p9[i]);
  else return f2_const(kLog1p7[i]);
}
// e^{-|z|}. For f32 tensors with what the product -|z| log2(e) rounds off (at z = 60 that is 2^-18 of
// the result; a 16-bit logit's own step is far coarser).
template <typename T>
__device__ __forceinline__ float exp_neg_abs(float z) {
  const float hi = -kLog2e * fabsf(z);
  if constexpr (sizeof(T) == 2) return ex2_approx(hi);
  const float lo = fmaf(-kLog2eLow, fabsf(z), fmaf(-kLog2e, fabsf(z), -hi)), e = ex2_approx(hi);
  return hi > -126.f ? fmaf(e, lo * kLn2, e) : e;  // also keeps inf - inf out
}
// softplus(-z) and e^{-|z|} of K pairs. The K are taken through every operation together: one pair's
// operations wait for each other, and a scheduler has few warps to fill the gaps.
template <typename T, int K>
__device__ __forceinline__ void softplus_neg(const uint64_t (&z)[K], uint64_t (&s)[K], uint64_t (&e)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float2 f = f2_unpack(z[k]);
    e[k] = f2_pack(exp_neg_abs<T>(f.x), exp_neg_abs<T>(f.y));
  }
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = log1p_term<T>(kDegree<T>);
#pragma unroll
  for (int i = kDegree<T> - 1; i >= 0; --i)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = f2_fma(s[k], e[k], log1p_term<T>(i));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float2 f = f2_unpack(z[k]);
    s[k] = f2_fma(e[k], s[k], f2_pack(fmaxf(-f.x, 0.f), fmaxf(-f.y, 0.f)));
  }
}
// e^{-S / tau} - 1 of K pairs by the expansion
template <typename T, int K>
__device__ __forceinline__ void expm1_small(const uint64_t (&s)[K], const DecayParams& g, uint64_t (&r)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) r[k] = f2_const(g.expm1[kExpDegree<T>]);
#pragma unroll
  for (int i = kExpDegree<T> - 1; i >= 0; --i)
#pragma unroll
    for (int k = 0; k < K; ++k) r[k] = f2_fma(r[k], s[k], f2_const(g.expm1[i]));
#pragma unroll
  for (int k = 0; k < K; ++k) r[k] = f2_mul(s[k], r[k]);
}
// 1 - sigmoid(z), given e = e^{-|z|} and r = 1 / (1 + e)
__device__ __forceinline__ uint64_t sigmoid_down(uint64_t z, uint64_t e, uint64_t r) {
  const float2 f = f2_unpack(z), g = f2_unpack(e);
  return f2_mul(f2_pack(f.x >= 0.f ? g.x : 1.f, f.y >= 0.f ? g.y : 1.f), r);
}
__device__ __forceinline__ uint64_t rcp_one_plus(uint64_t e) {
  const float2 f = f2_unpack(e);
  return f2_pack(rcp_approx(1.f + f.x), rcp_approx(1.f + f.y));
}

// -c of K pairs of logits. With S = softplus(-z), -c = e^{-S / tau} - 1 is S times a polynomial in S
// while S <= tau / 2; beyond (FAR: look for it), where e^{-S / tau} < 0.61 loses nothing in the
// difference from one, it is that difference. TAU1: c = 1 - sigmoid(z) in closed form.
// SLOPE: also -dc/dz = a (1 - sigmoid(z)) / tau, accurate relative to itself: for gates that forget a is
// not taken as 1 - c, which has lost it, but as the exponential that c came from, and with tau = 1 the
// slope is sigmoid(z) (1 - sigmoid(z)) = e / (1 + e)^2. For padded rows (z = +inf) both are zero.
template <typename T, bool TAU1, bool FAR, bool SLOPE, int K>
__device__ __forceinline__ void neg_decay(const uint64_t (&z)[K], const DecayParams& g, uint64_t (&nc)[K], uint64_t (&slope)[K]) {
  uint64_t e[K];
  if constexpr (TAU1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float2 f = f2_unpack(z[k]);
      e[k] = f2_pack(exp_neg_abs<T>(f.x), exp_neg_abs<T>(f.y));
      const uint64_t r = rcp_one_plus(e[k]);
      nc[k] = f2_neg(sigmoid_down(z[k], e[k], r));
      if (SLOPE) slope[k] = f2_mul(f2_mul(e[k], r), r);
    }
  } else {
    uint64_t s[K];
    softplus_neg<T>(z, s, e);
    expm1_small<T>(s, g, nc);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint64_t d = 0;
      if constexpr (SLOPE) {
        d = f2_mul(sigmoid_down(z[k], e[k], rcp_one_plus(e[k])), f2_both(g.inv_tau));
        slope[k] = f2_fma(nc[k], d, d);
      }
      if constexpr (FAR) {
        const float2 f = f2_unpack(s[k]), down = f2_unpack(d);
        float2 n = f2_unpack(nc[k]), v = SLOPE ? f2_unpack(slope[k]) : down;
        if (f.x > g.far) {
          const float a = ex2_approx(-kLog2e * g.inv_tau * f.x);
          n.x = a - 1.f, v.x = a * down.x;
        }
        if (f.y > g.far) {
          const float a = ex2_approx(-kLog2e * g.inv_tau * f.y);
          n.y = a - 1.f, v.y = a * down.y;
        }
        nc[k] = f2_pack(n.x, n.y);
        if (SLOPE) slope[k] = f2_pack(v.x, v.y);
      }
    }
  }
}

// Whether some of a warp's R rows of logits in shared memory has an S beyond the expansion: seen from
// the smallest logit, before anything is computed.
template <typename T, bool TAU1, int R>
__device__ __forceinline__ bool any_far(const typename Pair<T>::Raw* zs, const DecayParams& g) {
  using P = Pair<T>;
  if constexpr (TAU1) return false;
  typename P::Raw least = zs[0];
#pragma unroll
  for (int r = 1; r < R; ++r) least = P::least(least, zs[r * 32]);
  const float2 f = f2_unpack(P::f32(least));
  return fminf(f.x, f.y) < g.far_logit;
}

// -c of a warp's R rows of logits, kBatch pairs at a time.
constexpr int kBatch = 4;
template <typename T, bool TAU1, int R>
__device__ __forceinline__ void row_decays(const typename Pair<T>::Raw* zs, const DecayParams& g, uint64_t (&nc)[R]) {
  using P = Pair<T>;
  auto rows = [&](auto far) {
#pragma unroll
    for (int r = 0; r < R; r += kBatch) {
      uint64_t z[kBatch], v[kBatch], unused[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) z[k] = P::f32(zs[(r + k) * 32]);
      neg_decay<T, TAU1, decltype(far)::value, false>(z, g, v, unused);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) nc[r + k] = v[k];
    }
  };
  if (any_far<T, TAU1, R>(zs, g)) rows(std::true_type{});
  else rows(std::false_type{});
}

// h - c h + u, x as loaded
template <typename T, bool TIED>
__device__ __forceinline__ uint64_t advance(uint64_t h, uint64_t nc, typename Pair<T>::Raw x) {
  h = f2_fma(nc, h, h);
  return TIED ? f2_fma(nc, Pair<T>::minus(x), h) : f2_add(h, Pair<T>::f32(x));
}

// ---------------------------------------------------------------- values that are not finite
// h - c h is NaN for an infinite h, a h is infinite. Looking at every state would cost the sequence
// kernels issue slots in every row. But from an infinity or NaN on, a channel's values are infinite or
// NaN to the end (a padded row keeps them, a gate of zero makes them NaN) in the fast form as in the
// formula, so its last value tells: where that is not finite one warp computes the channel again, row by
// row with a h itself, when everything else of the tile has been stored. The other channels keep their bits.
// Such a tile takes about 0.3 us a row, its gradients 0.4 (8 x 2048 x 2048 bf16 with an infinity in every
// tile: 0.61 and 0.86 ms); tiles without one take what they took before this was looked at.
__device__ __forceinline__ uint32_t not_finite(uint64_t v, int n) {  // bit i: the i-th of n channels
  const float2 f = f2_unpack(v);
  return (n > 0 && !(fabsf(f.x) < INFINITY) ? 1u : 0u) | (n > 1 && !(fabsf(f.y) < INFINITY) ? 2u : 0u);
}
__device__ __forceinline__ void store_some(float* p, uint32_t which, uint64_t v) {
  const float2 f = f2_unpack(v);
  if (which & 1u) p[0] = f.x;
  if (which & 2u) p[1] = f.y;
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, uint32_t which, typename Pair<T>::Raw v) {
  if (which & 1u) p[0] = Pair<T>::half(v, 0);
  if (which & 2u) p[1] = Pair<T>::half(v, 1);
}
// a h for any h, given -c and whether a is zero (a logit of -inf; bit i: the i-th channel)
__device__ __forceinline__ uint32_t gate_zero(uint64_t z) {
  const float2 f = f2_unpack(z);
  return (f.x == -INFINITY ? 1u : 0u) | (f.y == -INFINITY ? 2u : 0u);
}
__device__ __forceinline__ float decayed(float h, float nc, bool zero) {
  if (fabsf(h) < INFINITY) return fmaf(nc, h, h);
  return zero ? NAN : h + nc;  // h, or NaN where the gate is
}
__device__ __forceinline__ uint64_t decayed(uint64_t h, uint64_t nc, uint32_t zero) {
  const float2 f = f2_unpack(h), c = f2_unpack(nc);
  return f2_pack(decayed(f.x, c.x, (zero & 1u) != 0), decayed(f.y, c.y, (zero & 2u) != 0));
}
template <typename T, bool TIED>
__device__ __forceinline__ uint64_t advance_any(uint64_t h, uint64_t nc, uint32_t zero, typename Pair<T>::Raw x) {
  h = decayed(h, nc, zero);
  return TIED ? f2_fma(nc, Pair<T>::minus(x), h) : f2_add(h, Pair<T>::f32(x));
}
// A row's factor of its gate's gradient, kept in the places of x and z.
template <typename T>
__device__ __forceinline__ void set_factor(typename Pair<T>::Raw* xs, typename Pair<T>::Raw* zs, uint64_t q) {
  if constexpr (sizeof(T) == 4) {
    *xs = q;
  } else {
    const float2 f = f2_unpack(q);
    *xs = __float_as_uint(f.x);
    *zs = __float_as_uint(f.y);
  }
}
template <typename T>
__device__ __forceinline__ uint64_t get_factor(const typename Pair<T>::Raw* xs, const typename Pair<T>::Raw* zs) {
  if constexpr (sizeof(T) == 4) return *xs;
  else return f2_pack(__uint_as_float(*xs), __uint_as_float(*zs));
}
template <bool TIED>
__device__ __forceinline__ uint64_t input_grad(uint64_t nc, uint64_t g) {
  return TIED ? f2_neg(f2_mul(nc, g)) : g;
}

// ---------------------------------------------------------------- blocks and clusters
// What a chunk hands over: the decay product and local end value of its rows.
struct alignas(16) Join {
  uint64_t p, v;
};

// Sends this block's join to every block of the cluster, and later waits for theirs. What the
// other warps read of the slots two steps ago is ordered before the sender's release by
// the block barrier between, so they need not release anything themselves.
__device__ __forceinline__ void send_join(Join* slots, int rank, int cluster, const Join& j, bool sender) {
  if (sender) {
    const uint32_t at = smem_u32(slots + rank * 32 + lane_id());
    for (int r = 0; r < cluster; ++r)
      asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(mapa_shared(at, r)), "l"(j.p), "l"(j.v) : "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  } else {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  }
}
__device__ __forceinline__ void receive_joins() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Joins a block's warps in their order: what comes before warp w, and all of them.
template <int WARPS>
__device__ __forceinline__ void join_warps(const Join (*wj)[32], int w, Join& before, Join& all) {
  before = all = Join{f2_both(1.f), 0ull};
#pragma unroll
  for (int j = 0; j < WARPS; ++j) {
    if (j == w) before = all;
    const Join q = wj[j][lane_id()];
    all.v = f2_fma(q.p, all.v, q.v);
    all.p = f2_mul(q.p, all.p);
  }
}
// The cluster's blocks in their order: returns what `carry` is before block `rank`, and takes
// `carry` past all of them.
__device__ __forceinline__ uint64_t pass_blocks(const Join* slots, int rank, int cluster, uint64_t& carry) {
  uint64_t mine = carry;
  for (int j = 0; j < cluster; ++j) {
    if (j == rank) mine = carry;
    const Join q = slots[j * 32 + lane_id()];
    carry = f2_fma(q.p, carry, q.v);
  }
  return mine;
}

// The valid rows of the chunks a warp takes one after another. The mask of a chunk decides which
// copies are started, so its bytes are loaded one chunk earlier still (the copies
// waited for them otherwise: 6 us of a forward of 8 x 2048 x 2048).
template <int R>
struct ValidRows {
  const uint8_t* mask;  // of the sequence, or null
  int L, ahead;
  __device__ __forceinline__ ValidRows(const ScanParams& p, int b) : mask(p.mask), L(p.L), ahead(0) {
    if (mask) mask += static_cast<size_t>(b) * L;
  }
  __device__ __forceinline__ void look(int t0) {  // rows t0 .. t0 + R - 1 come next
    const int t = t0 + lane_id();
    if (mask) ahead = lane_id() < R && t >= 0 && t < L ? mask[t] : 0;
  }
  // bit r: row t0 + r, the rows looked at last; then looks at those from `next` on
  __device__ __forceinline__ uint32_t take(int t0, int next) {
    if (!mask) {
      const int n = t0 < 0 ? 0 : min(max(L - t0, 0), R);
      return (1u << n) - 1u;
    }
    const uint32_t bits = __ballot_sync(~0u, ahead != 0);
    look(next);
    return bits;
  }
};

// ---------------------------------------------------------------- rows in shared memory

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a lane's part of a warp's rows stands: 16 bytes of every kEach-th row with VEC (rows
// aligned to 16 bytes, D a whole number of them), else the lane's pair of every row.
template <typename T, bool VEC>
struct Lane {
  static constexpr int kRow = 64 * sizeof(T), kEach = VEC ? 512 / kRow : 1;
  T* at;            // in the row given to go_to
  long long row;
  int first, n;     // its first row, its channels inside D
  __device__ __forceinline__ Lane(const Rows& r, int b, int c0, int D) {
    const int c = VEC ? lane_id() * 16 % kRow / static_cast<int>(sizeof(T)) : 2 * lane_id();
    first = VEC ? lane_id() * 16 / kRow : 0;
    n = min(max(D - c0 - c, 0), VEC ? 16 / static_cast<int>(sizeof(T)) : 2);
    row = r.row;
    at = static_cast<T*>(r.ptr) + b * r.batch + first * r.row + c0 + c;
  }
  __device__ __forceinline__ void move(long long rows) { at += rows * row; }
  // Without VEC: whether the lane's pair is one aligned word of 4 bytes (two of f32) in every row.
  __device__ __forceinline__ bool words() const {
    return sizeof(T) == 4 || (reinterpret_cast<uintptr_t>(at) % 4 == 0 && row % 2 == 0);
  }
};

// Starts a warp's copy of R rows to `to`; rows whose bit is not set and channels past D
// become `none`. full: every row is valid and every channel inside D. Without VEC the lanes copy
// their pairs word by word where they can, and load and store them at once where not (an
// odd number of 16-bit channels).
template <typename T, bool VEC>
__device__ __forceinline__ void fetch(uint8_t* to, const Lane<T, VEC>& l, bool full, uint32_t bits,
                                      typename Pair<T>::Raw none) {
  constexpr int R = kRowsOf<T>, kEach = Lane<T, VEC>::kEach;
  const T* from = l.at;
  const int lane = lane_id();
  if constexpr (VEC) {
    const uint32_t at = smem_u32(to) + lane * 16, v = static_cast<uint32_t>(none);  // a 64-bit pair's halves are alike
    if (full) {
#pragma unroll
      for (int i = 0; i < R / kEach; ++i, from += kEach * l.row) copy16(at + i * 512, from);
    } else {
      bits >>= l.first;
#pragma unroll
      for (int i = 0; i < R / kEach; ++i, from += kEach * l.row) {
        if (l.n && (bits >> i * kEach & 1)) copy16(at + i * 512, from);
        else st_shared_v4(at + i * 512, v, v, v, v);
      }
    }
  } else {
    using Raw = typename Pair<T>::Raw;
    Raw* at = reinterpret_cast<Raw*>(to) + lane;
    constexpr int kStep = Lane<T, VEC>::kRow / sizeof(Raw);
    if (sizeof(T) == 4) {
#pragma unroll 4
      for (int i = 0; i < R; ++i, from += l.row, at += kStep) {
        const int n = bits >> i & 1 ? l.n : 0;
        if (n == 0) *at = none;
        if (n == 1) reinterpret_cast<uint32_t*>(at)[1] = static_cast<uint32_t>(none);
        if (n > 0) copy4(smem_u32(at), from);
        if (n > 1) copy4(smem_u32(at) + 4, from + 1);
      }
    } else if (l.words()) {
#pragma unroll 4
      for (int i = 0; i < R; ++i, from += l.row, at += kStep) {
        const int n = bits >> i & 1 ? l.n : 0;
        if (n == 2) copy4(smem_u32(at), from);
        else *at = load_pair<T, false>(from, n, none);
      }
    } else {
#pragma unroll 8
      for (int i = 0; i < R; ++i, from += l.row) at[i * kStep] = load_pair<T, false>(from, bits >> i & 1 ? l.n : 0, none);
    }
  }
}

// Stores the first `rows` (1 .. R) of a warp's rows from shared memory; those whose bit is
// not set as zeros.
template <typename T, bool VEC>
__device__ __forceinline__ void put(const uint8_t* from, const Lane<T, VEC>& l, bool full, int rows, uint32_t bits) {
  constexpr int R = kRowsOf<T>, kEach = Lane<T, VEC>::kEach;
  const int lane = lane_id();
  T* to = l.at;
  if constexpr (VEC) {
    const uint4* v = reinterpret_cast<const uint4*>(from) + lane;
    if (full) {
#pragma unroll
      for (int i = 0; i < R / kEach; ++i, to += kEach * l.row) *reinterpret_cast<uint4*>(to) = v[i * 32];
    } else {
      bits >>= l.first;
      rows -= l.first;
#pragma unroll
      for (int i = 0; i < R / kEach; ++i, to += kEach * l.row)
        if (l.n && i * kEach < rows) *reinterpret_cast<uint4*>(to) = bits >> i * kEach & 1 ? v[i * 32] : make_uint4(0, 0, 0, 0);
    }
  } else {
    using Raw = typename Pair<T>::Raw;
    const Raw* v = reinterpret_cast<const Raw*>(from) + lane;
    const bool word = sizeof(T) == 2 && l.words() && l.n == 2;
#pragma unroll 4
    for (int i = 0; i < R; ++i, to += l.row, v += Lane<T, VEC>::kRow / sizeof(Raw))
      if (i < rows) {
        const Raw r = bits >> i & 1 ? *v : Pair<T>::zero();
        if (word) *reinterpret_cast<Raw*>(to) = r;
        else store_pair<T, false>(to, l.n, r);
      }
  }
}

// A warp's channels `bad` (a lane's bits 0 and 1: of its pair) of sequence b once more, from the first
// row (see "values that are not finite"). space: shared memory that no one else uses, a chunk of x and z.
// Both functions are compiled into every sequence kernel, so they are kept short: one chunk at a time, the
// general form of the gate for tau = 1 too.
template <typename T, bool TIED>
__device__ __noinline__ void forward_again(const ScanParams& p, int b, int c0, uint32_t bad, uint8_t* space) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int R = kRowsOf<T>;
  const int ch = c0 + 2 * lane_id(), n = min(max(p.D - ch, 0), 2), chunks = (p.L + R - 1) / R;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  const Raw* xs = reinterpret_cast<const Raw*>(space) + lane_id();
  T* out = static_cast<T*>(p.h.ptr) + b * p.h.batch + ch;
  Lane<T, false> lx(p.x, b, c0, p.D), lz(p.z, b, c0, p.D);
  ValidRows<R> valid(p, b);
  valid.look(0);
  uint64_t h = p.h0 ? load_state<false>(p.h0 + state_at, n) : 0ull;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const uint32_t bits = valid.take(c * R, (c + 1) * R);
    fetch<T, false>(space, lx, false, bits, P::zero());
    fetch<T, false>(space + kRowsBytes, lz, false, bits, P::inf());
    copies_commit();
    lx.move(R), lz.move(R);
    if (p.saved) store_some(p.saved + (static_cast<size_t>(b) * chunks + c) * p.D + ch, bad, h);
    copies_wait<0>();
    const int rows = min(p.L - c * R, R);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kBatch) {
      uint64_t z[kBatch], nc[kBatch], unused[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) z[k] = P::f32(xs[kRowsBytes / sizeof(Raw) + (r0 + k) * 32]);
      neg_decay<T, false, true, false>(z, p.gate, nc, unused);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        h = advance_any<T, TIED>(h, nc[k], gate_zero(z[k]), xs[(r0 + k) * 32]);
        if (r0 + k < rows) store_some<T>(out + k * p.h.row, bad, bits >> (r0 + k) & 1 ? P::round(h) : P::zero());
      }
      out += kBatch * p.h.row;
    }
  }
  store_some(p.last + state_at, bad, h);
}

// Their gradients, from the last row. space: a chunk of x, z and dh, and the rows' decays.
template <typename T, bool TIED>
__device__ __noinline__ void backward_again(const ScanParams& p, int b, int c0, uint32_t bad, uint8_t* space) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int R = kRowsOf<T>;
  const int ch = c0 + 2 * lane_id(), n = min(max(p.D - ch, 0), 2), chunks = (p.L + R - 1) / R;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  Raw* xs = reinterpret_cast<Raw*>(space) + lane_id();
  Raw* zs = xs + kRowsBytes / sizeof(Raw);
  const Raw* ds = zs + kRowsBytes / sizeof(Raw);
  uint64_t* ncs = reinterpret_cast<uint64_t*>(space + 3 * kRowsBytes) + lane_id();
  Lane<T, false> lx(p.x, b, c0, p.D), lz(p.z, b, c0, p.D), ld(p.dh, b, c0, p.D);
  lx.move((chunks - 1) * R), lz.move((chunks - 1) * R), ld.move((chunks - 1) * R);
  ValidRows<R> valid(p, b);
  valid.look((chunks - 1) * R);
  uint64_t in = p.dlast ? load_state<false>(p.dlast + state_at, n) : 0ull;
#pragma unroll 1
  for (int c = chunks - 1; c >= 0; --c) {
    const uint32_t bits = valid.take(c * R, (c - 1) * R);
    fetch<T, false>(space, lx, false, bits, P::zero());
    fetch<T, false>(space + kRowsBytes, lz, false, bits, P::inf());
    fetch<T, false>(space + 2 * kRowsBytes, ld, false, p.dh.ptr ? bits : 0u, P::zero());
    copies_commit();
    lx.move(-R), lz.move(-R), ld.move(-R);
    uint64_t h = load_state<false>(p.saved + (static_cast<size_t>(b) * chunks + c) * p.D + ch, n);
    copies_wait<0>();
    uint32_t zeros = 0;  // two bits a row: gates of zero
#pragma unroll 1
    for (int r0 = 0; r0 < R; r0 += kBatch) {
      uint64_t z[kBatch], nc[kBatch], slope[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) z[k] = P::f32(zs[(r0 + k) * 32]);
      neg_decay<T, false, true, true>(z, p.gate, nc, slope);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = r0 + k;
        const Raw x = xs[r * 32];
        set_factor<T>(xs + r * 32, zs + r * 32, f2_mul(TIED ? f2_add(h, P::minus(x)) : h, slope[k]));
        h = advance_any<T, TIED>(h, nc[k], gate_zero(z[k]), x);
        ncs[r * 32] = nc[k];
        zeros |= gate_zero(z[k]) << 2 * r;
      }
    }
    T* dx = static_cast<T*>(p.dx.ptr) + b * p.dx.batch + (static_cast<long long>(c) * R + R - 1) * p.dx.row + ch;
    T* dz = static_cast<T*>(p.dz.ptr) + b * p.dz.batch + (static_cast<long long>(c) * R + R - 1) * p.dz.row + ch;
#pragma unroll 1
    for (int r = R - 1; r >= 0; --r, dx -= p.dx.row, dz -= p.dz.row) {
      const uint64_t nc = ncs[r * 32], q = get_factor<T>(xs + r * 32, zs + r * 32), g = f2_add(in, P::f32(ds[r * 32]));
      in = decayed(g, nc, zeros >> 2 * r & 3u);
      if (bits >> r & 1) {  // padded rows and those past the end are as they should be
        store_some<T>(dx, bad, P::round(input_grad<TIED>(nc, g)));
        store_some<T>(dz, bad, P::round(f2_mul(g, q)));
      }
    }
  }
  if (p.dh0) store_some(p.dh0 + state_at, bad, in);
}

// ---------------------------------------------------------------- forward, rows split over a cluster
// Every step takes cluster x kWarps chunks. The next step's gates and local results are made between
// sending a step's joins and waiting for the other blocks'.
constexpr int kWarps = 16;
constexpr int kSlots = 2 * 32 * sizeof(Join);  // what one block of a cluster sends, double-buffered
constexpr int kForwardRows = kWarps * 3 * 2 * kRowsBytes;  // three steps: two used, one on its way

template <typename T, bool VEC, bool TAU1, bool TIED>
__global__ void __launch_bounds__(kWarps * 32, 1) scan_forward_kernel(const __grid_constant__ ScanParams p) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int R = kRowsOf<T>, kRows = kWarps * R;
  extern __shared__ __align__(128) uint8_t dynamic[];
  __shared__ Join warps[2][kWarps][32];
  const int cluster = p.cluster, rank = cluster_ctarank();
  const int w = warp_id(), lane = lane_id(), b = blockIdx.y;
  const int c0 = blockIdx.x / cluster * 64, ch = c0 + 2 * lane, n = min(max(p.D - ch, 0), 2);
  uint8_t* mine = dynamic + w * 3 * 2 * kRowsBytes;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  const int chunks = (p.L + R - 1) / R, steps = (p.L + cluster * kRows - 1) / (cluster * kRows);
  const bool inside = c0 + 64 <= p.D;
  Lane<T, VEC> lx(p.x, b, c0, p.D), lz(p.z, b, c0, p.D), lo(p.h, b, c0, p.D);
  const int first = (rank * kWarps + w) * R;
  lx.move(first), lz.move(first), lo.move(first);
  ValidRows<R> valid(p, b);
  valid.look(first);
  auto start_step = [&](int step) {
    uint32_t bits = 0;
    if (step < steps) {
      uint8_t* to = mine + step % 3 * 2 * kRowsBytes;
      bits = valid.take(first + step * cluster * kRows, first + (step + 1) * cluster * kRows);
      const bool full = inside && bits == (1u << R) - 1u;
      fetch<T, VEC>(to, lx, full, bits, P::zero());
      fetch<T, VEC>(to + kRowsBytes, lz, full, bits, P::inf());
      lx.move(cluster * kRows), lz.move(cluster * kRows);
    }
    copies_commit();
    return bits;
  };
  auto rows_of = [&](int step) { return reinterpret_cast<Raw*>(mine + step % 3 * 2 * kRowsBytes) + lane; };
  auto local = [&](int step, uint64_t (&nc)[R]) {
    copies_wait<1>();
    __syncwarp();
    const Raw* xs = rows_of(step);
    row_decays<T, TAU1>(xs + kRowsBytes / sizeof(Raw), p.gate, nc);
    Join join{f2_both(1.f), 0ull};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      join.v = advance<T, TIED>(join.v, nc[r], xs[r * 32]);
      join.p = f2_fma(nc[r], join.p, join.p);
    }
    warps[step & 1][w][lane] = join;
  };

  uint32_t now = start_step(0), next = start_step(1);
  uint64_t carry = p.h0 ? load_state<VEC>(p.h0 + state_at, n) : 0ull;
  cluster_sync();  // every block runs before another writes to it
  uint64_t nc[R], nc_next[R];
  local(0, nc);
  for (int step = 0; step < steps; ++step) {
    const int t0 = first + step * cluster * kRows;
    __syncthreads();
    Join before, all;
    join_warps<kWarps>(warps[step & 1], w, before, all);
    Join* slots = reinterpret_cast<Join*>(dynamic + kForwardRows) + (step & 1) * cluster * 32;
    send_join(slots, rank, cluster, all, w == 0);
    const uint32_t after = start_step(step + 2);
    if (step + 1 < steps) local(step + 1, nc_next);
    receive_joins();
    uint64_t h = pass_blocks(slots, rank, cluster, carry);
    h = f2_fma(before.p, h, before.v);
    if (p.saved && t0 < p.L) store_state<VEC>(p.saved + (static_cast<size_t>(b) * chunks + t0 / R) * p.D + ch, n, h);
    Raw* xs = rows_of(step);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h = advance<T, TIED>(h, nc[r], xs[r * 32]);
      xs[r * 32] = P::round(h);
      nc[r] = nc_next[r];
    }
    __syncwarp();
    if (t0 < p.L) put<T, VEC>(mine + step % 3 * 2 * kRowsBytes, lo, inside && now == (1u << R) - 1u, min(p.L - t0, R), now);
    lo.move(cluster * kRows);
    __syncwarp();
    now = next;
    next = after;
  }
  const bool ends = rank == 0 && w == 0;
  const uint32_t bad = not_finite(carry, n);  // the same in every warp of the cluster: all have joined the same values
  if (ends && !bad) store_state<VEC>(p.last + state_at, n, carry);
  if (ends && bad) store_some(p.last + state_at, ~bad & ((1u << n) - 1u), carry);
  if (__any_sync(~0u, bad)) {
    cluster_sync();  // every block's rows are stored
    if (ends) forward_again<T, TIED>(p, b, c0, bad, dynamic);
  }
}

// ---------------------------------------------------------------- forward, one block per tile
// The block's warps take the chunks of R rows in turn, each on its own: copies, gate, the
// chunk's decay product and local end state. Only the true state goes from warp to warp in
// the chunks' order, a relay with one named barrier a warp: a hop is one product and sum, and
// the rows of a chunk follow from the state before it while the next warps go on.
__device__ __forceinline__ void relay_wait(int warp) { asm volatile("bar.sync %0, 64;" ::"r"(1 + warp) : "memory"); }
__device__ __forceinline__ void relay_pass(int warp) { asm volatile("bar.arrive %0, 64;" ::"r"(1 + warp) : "memory"); }

constexpr int kRelay = 12;  // warps of a block
constexpr int kRelayShared = kRelay * 2 * 2 * kRowsBytes;

template <typename T, bool VEC, bool TAU1, bool TIED>
__global__ void __launch_bounds__(kRelay * 32, 2) scan_relay_kernel(const __grid_constant__ ScanParams p) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int R = kRowsOf<T>;
  constexpr uint32_t kFull = (1u << R) - 1u;
  extern __shared__ __align__(128) uint8_t dynamic[];
  __shared__ uint64_t baton[kRelay][32];
  const int w = warp_id(), lane = lane_id(), b = blockIdx.y, c0 = blockIdx.x * 64;
  const int ch = c0 + 2 * lane, n = min(max(p.D - ch, 0), 2);
  const int chunks = (p.L + R - 1) / R;
  const bool inside = c0 + 64 <= p.D;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  uint8_t* mine = dynamic + w * 4 * kRowsBytes;
  float* saved = p.saved ? p.saved + (static_cast<size_t>(b) * chunks + w) * p.D + ch : nullptr;
  Lane<T, VEC> lx(p.x, b, c0, p.D), lz(p.z, b, c0, p.D), lo(p.h, b, c0, p.D);
  lx.move(w * R), lz.move(w * R), lo.move(w * R);
  ValidRows<R> valid(p, b);
  valid.look(w * R);
  auto start = [&](int c, int slot) {
    uint32_t bits = 0;
    if (c < chunks) {
      uint8_t* to = mine + slot * 2 * kRowsBytes;
      bits = valid.take(c * R, (c + kRelay) * R);
      const bool full = inside && bits == kFull;
      fetch<T, VEC>(to, lx, full, bits, P::zero());
      fetch<T, VEC>(to + kRowsBytes, lz, full, bits, P::inf());
      lx.move(kRelay * R), lz.move(kRelay * R);
    }
    copies_commit();
    return bits;
  };
  uint32_t now = start(w, 0), bad = 0;
  for (int c = w, slot = 0; c < chunks; c += kRelay, slot ^= 1) {
    const uint32_t next = start(c + kRelay, slot ^ 1);
    copies_wait<1>();
    __syncwarp();
    uint8_t* rows = mine + slot * 2 * kRowsBytes;
    Raw* xs = reinterpret_cast<Raw*>(rows) + lane;
    uint64_t nc[R];
    row_decays<T, TAU1>(xs + kRowsBytes / sizeof(Raw), p.gate, nc);
    Join join{f2_both(1.f), 0ull};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      join.v = advance<T, TIED>(join.v, nc[r], xs[r * 32]);
      join.p = f2_fma(nc[r], join.p, join.p);
    }
    uint64_t h;
    if (c == 0) {
      h = p.h0 ? load_state<VEC>(p.h0 + state_at, n) : 0ull;
    } else {
      relay_wait(w);
      h = baton[w][lane];
    }
    const uint64_t end = f2_fma(join.p, h, join.v);
    if (c + 1 < chunks) {
      const int to = w + 1 == kRelay ? 0 : w + 1;
      baton[to][lane] = end;
      relay_pass(to);
    } else {
      bad = not_finite(end, n);
      if (!bad) store_state<VEC>(p.last + state_at, n, end);
      else store_some(p.last + state_at, ~bad & ((1u << n) - 1u), end);
    }
    if (saved) {
      store_state<VEC>(saved, n, h);
      saved += static_cast<size_t>(kRelay) * p.D;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      h = advance<T, TIED>(h, nc[r], xs[r * 32]);
      xs[r * 32] = P::round(h);
    }
    __syncwarp();
    put<T, VEC>(rows, lo, inside && now == kFull, min(p.L - c * R, R), now);
    lo.move(kRelay * R);
    __syncwarp();
    now = next;
  }
  if (__syncthreads_or(bad) && __any_sync(~0u, bad)) forward_again<T, TIED>(p, b, c0, bad, dynamic);
}

// ---------------------------------------------------------------- backward
// Chunks of R rows, from the last. A chunk's states are rebuilt from its saved one, so
// everything but g is independent of the other chunks: per row -c and
// q = (h_{t-1} - [tied] x_t) a_t (1 - sigmoid(z_t)) / tau. Then, down the rows,
// g_t = dh_t + in, dz_t = g_t q_t, in = a_t g_t. q takes the place of x and z in shared
// memory (with -c and q of 16 rows in registers, 64 of them, the kernels spilled). Returns the state
// after the rows.
template <typename T, bool TAU1, bool TIED>
__device__ __forceinline__ uint64_t row_factors(typename Pair<T>::Raw* xs, typename Pair<T>::Raw* zs, uint64_t h,
                                            const DecayParams& gate, uint64_t (&nc)[kRowsOf<T>]) {
  using P = Pair<T>;
  constexpr int R = kRowsOf<T>;
  auto rows = [&](auto far) {
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += kBatch) {
      uint64_t z[kBatch], v[kBatch], slope[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) z[k] = P::f32(zs[(r0 + k) * 32]);
      neg_decay<T, TAU1, decltype(far)::value, true>(z, gate, v, slope);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = r0 + k;
        const typename P::Raw x = xs[r * 32];
        const uint64_t q = f2_mul(TIED ? f2_add(h, P::minus(x)) : h, slope[k]);
        h = advance<T, TIED>(h, v[k], x);
        nc[r] = v[k];
        set_factor<T>(xs + r * 32, zs + r * 32, q);
      }
    }
  };
  if (any_far<T, TAU1, R>(zs, gate)) rows(std::true_type{});
  else rows(std::false_type{});
  return h;
}
// One block per tile, as the forward, with the chunks from the last and the relay going that
// way: a chunk hands down out = P in + G.
constexpr int kBackRelay = 8;
constexpr int kBackRelayShared = kBackRelay * 2 * 3 * kRowsBytes;

template <typename T, bool VEC, bool TAU1, bool TIED>
__global__ void __launch_bounds__(kBackRelay * 32, 2) scan_relay_backward_kernel(const __grid_constant__ ScanParams p) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int R = kRowsOf<T>;
  constexpr uint32_t kFull = (1u << R) - 1u;
  extern __shared__ __align__(128) uint8_t dynamic[];
  __shared__ uint64_t baton[kBackRelay][32];
  __shared__ uint64_t ends[32];  // the state after the last row
  const int w = warp_id(), lane = lane_id(), b = blockIdx.y, c0 = blockIdx.x * 64;
  const int ch = c0 + 2 * lane, n = min(max(p.D - ch, 0), 2);
  const int chunks = (p.L + R - 1) / R;
  const bool inside = c0 + 64 <= p.D;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  uint8_t* mine = dynamic + w * 6 * kRowsBytes;
  Lane<T, VEC> lx(p.x, b, c0, p.D), lz(p.z, b, c0, p.D), ld(p.dh, b, c0, p.D), ox(p.dx, b, c0, p.D), oz(p.dz, b, c0, p.D);
  const int first = (chunks - 1 - w) * R;  // below zero where the warp has no chunk: then it is not used
  lx.move(first), lz.move(first), ld.move(first), ox.move(first), oz.move(first);
  ValidRows<R> valid(p, b);
  valid.look(first);
  uint64_t state = 0ull;
  auto start = [&](int c, int slot) {
    uint32_t bits = 0;
    if (c >= 0) {
      uint8_t* to = mine + slot * 3 * kRowsBytes;
      bits = valid.take(c * R, (c - kBackRelay) * R);
      const bool full = inside && bits == kFull;
      fetch<T, VEC>(to, lx, full, bits, P::zero());
      fetch<T, VEC>(to + kRowsBytes, lz, full, bits, P::inf());
      fetch<T, VEC>(to + 2 * kRowsBytes, ld, full && p.dh.ptr, p.dh.ptr ? bits : 0u, P::zero());
      lx.move(-kBackRelay * R), lz.move(-kBackRelay * R), ld.move(-kBackRelay * R);
      state = load_state<VEC>(p.saved + (static_cast<size_t>(b) * chunks + c) * p.D + ch, n);
    }
    copies_commit();
    return bits;
  };
  uint32_t now = start(chunks - 1 - w, 0), bad = 0;
  for (int c = chunks - 1 - w, slot = 0; c >= 0; c -= kBackRelay, slot ^= 1) {
    const uint64_t before = state;
    const uint32_t next = start(c - kBackRelay, slot ^ 1);
    copies_wait<1>();
    __syncwarp();
    uint8_t* rows = mine + slot * 3 * kRowsBytes;
    Raw* xs = reinterpret_cast<Raw*>(rows) + lane;
    Raw* zs = xs + kRowsBytes / sizeof(Raw);
    const Raw* ds = zs + kRowsBytes / sizeof(Raw);
    uint64_t nc[R];
    const uint64_t after = row_factors<T, TAU1, TIED>(xs, zs, before, p.gate, nc);
    if (c == chunks - 1) ends[lane] = after;
    Join join{f2_both(1.f), 0ull};
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      join.v = f2_add(join.v, P::f32(ds[r * 32]));
      join.v = f2_fma(nc[r], join.v, join.v);
      join.p = f2_fma(nc[r], join.p, join.p);
    }
    uint64_t in;
    if (c == chunks - 1) {
      in = p.dlast ? load_state<VEC>(p.dlast + state_at, n) : 0ull;
    } else {
      relay_wait(w);
      in = baton[w][lane];
    }
    const uint64_t end = f2_fma(join.p, in, join.v);
    if (c > 0) {
      const int to = w + 1 == kBackRelay ? 0 : w + 1;
      baton[to][lane] = end;
      relay_pass(to);
    } else {
      bad = not_finite(end, n) | not_finite(ends[lane], n);
      if (p.dh0) {
        if (!bad) store_state<VEC>(p.dh0 + state_at, n, end);
        else store_some(p.dh0 + state_at, ~bad & ((1u << n) - 1u), end);
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const uint64_t g = f2_add(in, P::f32(ds[r * 32])), q = get_factor<T>(xs + r * 32, zs + r * 32);
      in = f2_fma(nc[r], g, g);
      xs[r * 32] = P::round(input_grad<TIED>(nc[r], g));
      zs[r * 32] = P::round(f2_mul(g, q));
    }
    __syncwarp();
    const bool full = inside && now == kFull;
    const int rows_in = min(p.L - c * R, R);
    put<T, VEC>(rows, ox, full, rows_in, now);
    put<T, VEC>(rows + kRowsBytes, oz, full, rows_in, now);
    ox.move(-kBackRelay * R), oz.move(-kBackRelay * R);
    __syncwarp();
    now = next;
  }
  if (__syncthreads_or(bad) && __any_sync(~0u, bad)) backward_again<T, TIED>(p, b, c0, bad, dynamic);
}

// Rows split over a cluster, as in the forward: rank 0 and its warp 0 take the latest chunks.
constexpr int kBackWarps = 11;  // three steps of x, z and dh fill the shared memory
constexpr int kBackRows = kBackWarps * 3 * 3 * kRowsBytes;

template <typename T, bool VEC, bool TAU1, bool TIED>
__global__ void __launch_bounds__(kBackWarps * 32, 1) scan_backward_kernel(const __grid_constant__ ScanParams p) {
  using P = Pair<T>;
  using Raw = typename P::Raw;
  constexpr int R = kRowsOf<T>;
  extern __shared__ __align__(128) uint8_t dynamic[];
  __shared__ Join warps[2][kBackWarps][32];
  __shared__ uint32_t last_bad[32];  // lanes' channels whose last state is not finite
  const int cluster = p.cluster, rank = cluster_ctarank();
  const int w = warp_id(), lane = lane_id(), b = blockIdx.y;
  const int c0 = blockIdx.x / cluster * 64, ch = c0 + 2 * lane, n = min(max(p.D - ch, 0), 2);
  uint8_t* mine = dynamic + w * 3 * 3 * kRowsBytes;
  const size_t state_at = static_cast<size_t>(b) * p.D + ch;
  const int chunks = (p.L + R - 1) / R, each = cluster * kBackWarps, steps = (chunks + each - 1) / each;
  const float* saved = p.saved + static_cast<size_t>(b) * chunks * p.D + ch;
  const bool inside = c0 + 64 <= p.D;
  Lane<T, VEC> lx(p.x, b, c0, p.D), lz(p.z, b, c0, p.D), ld(p.dh, b, c0, p.D), ox(p.dx, b, c0, p.D), oz(p.dz, b, c0, p.D);
  const int last = chunks - 1 - (rank * kBackWarps + w), back = -each * R;  // this warp's chunk of step 0
  lx.move(last * R), lz.move(last * R), ld.move(last * R), ox.move(last * R), oz.move(last * R);
  ValidRows<R> valid(p, b);
  valid.look(last * R);
  struct Step {
    uint32_t bits;
    uint64_t state;
  };
  auto start_step = [&](int step) {
    const int c = last - step * each;
    Step s{0, 0ull};
    if (step < steps) {  // with c < 0 no row is valid and nothing is read
      s.bits = valid.take(c * R, c * R + back);
      uint8_t* to = mine + step % 3 * 3 * kRowsBytes;
      const bool full = inside && s.bits == (1u << R) - 1u;
      fetch<T, VEC>(to, lx, full, s.bits, P::zero());
      fetch<T, VEC>(to + kRowsBytes, lz, full, s.bits, P::inf());
      fetch<T, VEC>(to + 2 * kRowsBytes, ld, full && p.dh.ptr, p.dh.ptr ? s.bits : 0u, P::zero());
      lx.move(back), lz.move(back), ld.move(back);
      if (c >= 0) s.state = load_state<VEC>(saved + static_cast<size_t>(c) * p.D, n);
    }
    copies_commit();
    return s;
  };
  auto rows_of = [&](int step) { return reinterpret_cast<Raw*>(mine + step % 3 * 3 * kRowsBytes) + lane; };
  constexpr int kTensor = kRowsBytes / sizeof(Raw);
  auto local = [&](int step, uint64_t state, uint64_t (&nc)[R]) {
    copies_wait<1>();
    __syncwarp();
    Raw* xs = rows_of(step);
    const uint64_t after = row_factors<T, TAU1, TIED>(xs, xs + kTensor, state, p.gate, nc);
    Join join{f2_both(1.f), 0ull};
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      join.v = f2_add(join.v, P::f32(xs[2 * kTensor + r * 32]));
      join.v = f2_fma(nc[r], join.v, join.v);
      join.p = f2_fma(nc[r], join.p, join.p);
    }
    warps[step & 1][w][lane] = join;
    return after;
  };

  Step now = start_step(0), next = start_step(1);
  uint64_t carry = p.dlast ? load_state<VEC>(p.dlast + state_at, n) : 0ull;
  cluster_sync();
  uint64_t nc[R], nc_next[R];
  const uint32_t state_bad = not_finite(local(0, now.state, nc), n);
  if (rank == 0 && w == 0)  // it has the sequence's last state; sent to the blocks with the first step's joins
    for (int r = 0; r < cluster; ++r) st_cluster_u32(mapa_shared(smem_u32(last_bad + lane), r), state_bad);
  for (int step = 0; step < steps; ++step) {
    const int c = last - step * each;
    __syncthreads();
    Join before, all;
    join_warps<kBackWarps>(warps[step & 1], w, before, all);
    Join* slots = reinterpret_cast<Join*>(dynamic + kBackRows) + (step & 1) * cluster * 32;
    send_join(slots, rank, cluster, all, w == 0);
    const Step after = start_step(step + 2);
    if (step + 1 < steps) local(step + 1, next.state, nc_next);
    receive_joins();
    uint64_t in = pass_blocks(slots, rank, cluster, carry);
    in = f2_fma(before.p, in, before.v);
    Raw* xs = rows_of(step);
    Raw* zs = xs + kTensor;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const uint64_t g = f2_add(in, P::f32(xs[2 * kTensor + r * 32])), q = get_factor<T>(xs + r * 32, zs + r * 32);
      in = f2_fma(nc[r], g, g);
      xs[r * 32] = P::round(input_grad<TIED>(nc[r], g));
      zs[r * 32] = P::round(f2_mul(g, q));
      nc[r] = nc_next[r];
    }
    __syncwarp();
    if (c >= 0) {
      const bool full = inside && now.bits == (1u << R) - 1u;
      const uint8_t* rows = mine + step % 3 * 3 * kRowsBytes;
      put<T, VEC>(rows, ox, full, min(p.L - c * R, R), now.bits);
      put<T, VEC>(rows + kRowsBytes, oz, full, min(p.L - c * R, R), now.bits);
    }
    ox.move(back), oz.move(back);
    __syncwarp();
    now = next;
    next = after;
  }
  const bool ends = rank == 0 && w == 0;
  const uint32_t bad = not_finite(carry, n) | last_bad[lane];  // the same in every warp of the cluster, as in the forward
  if (p.dh0 && ends && !bad) store_state<VEC>(p.dh0 + state_at, n, carry);
  if (p.dh0 && ends && bad) store_some(p.dh0 + state_at, ~bad & ((1u << n) - 1u), carry);
  if (__any_sync(~0u, bad)) {
    cluster_sync();  // every block's rows are stored
    if (ends) backward_again<T, TIED>(p, b, c0, bad, dynamic);
  }
}

// ---------------------------------------------------------------- single tokens
template <typename T, bool VEC, bool TAU1, bool TIED>
__global__ void __launch_bounds__(128) scan_step_kernel(const StepParams p) {
  using P = Pair<T>;
  const int ch = (blockIdx.x * 128 + threadIdx.x) * 2, n = min(max(p.D - ch, 0), 2), b = blockIdx.y;
  if (n == 0) return;
  typename P::Raw out = P::zero();
  if (!p.mask || p.mask[b]) {
    float* s = p.state + static_cast<size_t>(b) * p.D + ch;
    const uint64_t z = P::f32(load_pair<T, VEC>(static_cast<const T*>(p.z) + b * p.z_row + ch, n, P::inf()));
    const typename P::Raw x = load_pair<T, VEC>(static_cast<const T*>(p.x) + b * p.x_row + ch, n, P::zero());
    const uint64_t zz[1] = {z};
    uint64_t nc[1], unused[1];
    neg_decay<T, TAU1, true, false>(zz, p.gate, nc, unused);
    const uint64_t h = advance_any<T, TIED>(load_state<VEC>(s, n), nc[0], gate_zero(z), x);
    store_state<VEC>(s, n, h);
    out = P::round(h);
  }
  store_pair<T, VEC>(static_cast<T*>(p.h) + b * p.h_row + ch, n, out);
}

// ---------------------------------------------------------------- launches
// f(element type, VEC, TAU1, TIED) with the values as compile-time constants
template <typename F>
void by_kind(int dtype, bool vec, bool tau1, bool tied, F&& f) {
  auto pick = [](bool v, auto&& g) {
    if (v) g(std::true_type{});
    else g(std::false_type{});
  };
  auto by_type = [&](auto t) {
    pick(vec, [&](auto v) { pick(tau1, [&](auto u) { pick(tied, [&](auto i) { f(t, v, u, i); }); }); });
  };
  if (dtype == kBF16) by_type(__nv_bfloat16{});
  else if (dtype == kF16) by_type(__half{});
  else by_type(float{});
}

// Whether runs of `run` channels from a multiple of `run` on are aligned in every row of r.
bool aligned_rows(const Rows& r, int run, int dtype) {
  const uintptr_t bytes = run * (dtype == kF32 ? 4 : 2);
  return !r.ptr || (reinterpret_cast<uintptr_t>(r.ptr) % bytes == 0 && r.batch % run == 0 && r.row % run == 0);
}
bool aligned_state(const float* s) { return reinterpret_cast<uintptr_t>(s) % 8 == 0; }

// Clusters of 2 .. kMaxCluster blocks of a split-rows kernel that run at once on the current device
// (its blocks fill an SM, and a cluster stays inside one of the GPU's SM groups: on a B200 74,
// .. 33 of 4, .. 15 of 8), asked for once a device.
template <int KIND>  // 0: forward, 1: backward
const int* clusters_at_once(const void* kernel, int threads, int shared) {
  constexpr int kDevices = 64;
  static int table[kDevices][kMaxCluster + 1];
  static std::once_flag once[kDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
  std::call_once(once[dev], [&] {
    for (int c = 2; c <= kMaxCluster; ++c) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = shared;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = c;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();  // the call's own launch is what reports an error
        n = 1;
      }
      table[dev][c] = n;
    }
  });
  return table[dev];
}

// Whether one block per channel tile and sequence is the form to take, or its rows are split over a
// cluster. A block of the first form keeps its SM busy by itself (9.5 ns a row of 64
// channels), one of the second at half that rate or more: where two blocks a tile find an
// SM each they win (8 tiles of 16384 rows: 37 us against 156, 64 tiles with gradients 333
// against 519), unless the rows are few (256 rows: 5.8 us against 5.3, 1024: 7.4 against 12.7).
bool one_block(long long tiles, int L, int rows, int pairs) { return tiles > pairs || L <= 2 * rows; }

// Blocks of a cluster, two at least: the fewest waves times steps, and of those the fewest blocks.
int pick_cluster(long long tiles, int L, int rows, const int* at_once) {
  int best = 2;
  long long least = 0;
  for (int c = 2; c <= kMaxCluster; ++c) {
    const long long time = (tiles + at_once[c] - 1) / at_once[c] * ((L + static_cast<long long>(c) * rows - 1) / (static_cast<long long>(c) * rows));
    if (c == 2 || time < least) best = c, least = time;
  }
  return best;
}

// (e^{-s} - 1) / s on [0, 1/2]: Chebyshev expansions cut off at degree 4 for 16-bit tensors
// (relative error 6e-8) and 5 for f32 (1e-9), with the powers of 1 / tau in the coefficients.
DecayParams decay_params(float inv_tau, int dtype) {
  constexpr double k4[6] = {-0.99999994, 0.4999924, -0.166547343, 0.0409987494, -0.0067685456, 0};
  constexpr double k5[6] = {-0.999999998605, 0.499999805417, -0.166662209042, 0.0416289147095, -0.00818699328274, 0.00112132441342};
  DecayParams g;
  g.inv_tau = inv_tau;
  g.far = 0.5f / inv_tau;
  // softplus(-z) = far at z = -log(e^far - 1), written without e^far: that overflows from tau = 1420 on, and
  // with a threshold of -inf no logit at all would be taken out of the expansion's range
  const double far = 0.5 / inv_tau;
  g.far_logit = static_cast<float>(-(far + std::log(-std::expm1(-far))));
  double power = inv_tau;
  for (int i = 0; i < 6; ++i, power *= inv_tau) {
    const float v = static_cast<float>((dtype == kF32 ? k5 : k4)[i] * power);
    g.expm1[i] = make_float2(v, v);
  }
  return g;
}

template <auto kernel>
cudaError_t launch(const ScanParams& p, int threads, int shared, cudaStream_t st) {
  const cudaError_t e = allow_shared<kernel>(shared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.D + 63) / 64 * p.cluster, p.B);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
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

int scan_saved_rows(int dtype) { return dtype == kF32 ? kRowsOf<float> : kRowsOf<__half>; }

cudaError_t launch_scan_forward(const ScanParams& params, cudaStream_t st) {
  ScanParams p = params;
  p.gate = decay_params(p.inv_tau, p.dtype);
  const int run = p.dtype == kF32 ? 4 : 8;
  const bool vec = p.D % run == 0 && aligned_rows(p.x, run, p.dtype) && aligned_rows(p.z, run, p.dtype) &&
                   aligned_rows(p.h, run, p.dtype) && aligned_state(p.h0) && aligned_state(p.last) && aligned_state(p.saved);
  const long long tiles = (p.D + 63LL) / 64 * p.B;
  cudaError_t e = cudaSuccess;
  by_kind(p.dtype, vec, p.inv_tau == 1.f, p.tied, [&](auto t, auto v, auto u, auto i) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value, U = decltype(u)::value, I = decltype(i)::value;
    constexpr int kRowsAtOnce = kWarps * kRowsOf<T>, kShared = kForwardRows + kMaxCluster * kSlots;
    e = allow_shared<scan_forward_kernel<T, V, U, I>>(kShared);
    if (e != cudaSuccess) return;
    const int* at_once = clusters_at_once<0>(reinterpret_cast<const void*>(scan_forward_kernel<T, V, U, I>), kWarps * 32, kShared);
    if (one_block(tiles, p.L, kRowsAtOnce, at_once[2])) {
      p.cluster = 1;
      e = launch<scan_relay_kernel<T, V, U, I>>(p, kRelay * 32, kRelayShared, st);
    } else {
      p.cluster = pick_cluster(tiles, p.L, kRowsAtOnce, at_once);
      e = launch<scan_forward_kernel<T, V, U, I>>(p, kWarps * 32, kShared, st);
    }
  });
  return e;
}

cudaError_t launch_scan_backward(const ScanParams& params, cudaStream_t st) {
  ScanParams p = params;
  p.gate = decay_params(p.inv_tau, p.dtype);
  const int run = p.dtype == kF32 ? 4 : 8;
  const bool vec = p.D % run == 0 && aligned_rows(p.x, run, p.dtype) && aligned_rows(p.z, run, p.dtype) &&
                   aligned_rows(p.dh, run, p.dtype) && aligned_rows(p.dx, run, p.dtype) &&
                   aligned_rows(p.dz, run, p.dtype) && aligned_state(p.saved) && aligned_state(p.dlast) &&
                   aligned_state(p.dh0);
  const long long tiles = (p.D + 63LL) / 64 * p.B;
  cudaError_t e = cudaSuccess;
  by_kind(p.dtype, vec, p.inv_tau == 1.f, p.tied, [&](auto t, auto v, auto u, auto i) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value, U = decltype(u)::value, I = decltype(i)::value;
    constexpr int kRowsAtOnce = kBackWarps * kRowsOf<T>, kShared = kBackRows + kMaxCluster * kSlots;
    e = allow_shared<scan_backward_kernel<T, V, U, I>>(kShared);
    if (e != cudaSuccess) return;
    const int* at_once = clusters_at_once<1>(reinterpret_cast<const void*>(scan_backward_kernel<T, V, U, I>), kBackWarps * 32, kShared);
    if (one_block(tiles, p.L, kRowsAtOnce, at_once[2])) {
      p.cluster = 1;
      e = launch<scan_relay_backward_kernel<T, V, U, I>>(p, kBackRelay * 32, kBackRelayShared, st);
    } else {
      p.cluster = pick_cluster(tiles, p.L, kRowsAtOnce, at_once);
      e = launch<scan_backward_kernel<T, V, U, I>>(p, kBackWarps * 32, kShared, st);
    }
  });
  return e;
}

cudaError_t launch_scan_step(const StepParams& params, cudaStream_t st) {
  StepParams p = params;
  p.gate = decay_params(p.inv_tau, p.dtype);
  const Rows rows[3] = {{const_cast<void*>(p.x), p.x_row, 0}, {const_cast<void*>(p.z), p.z_row, 0}, {p.h, p.h_row, 0}};
  bool vec = p.D % 2 == 0 && aligned_state(p.state);
  for (const Rows& r : rows) vec = vec && aligned_rows(r, 2, p.dtype);
  const dim3 grid((p.D + 255) / 256, p.B);
  cudaError_t e = cudaSuccess;
  by_kind(p.dtype, vec, p.inv_tau == 1.f, p.tied, [&](auto t, auto v, auto tau1, auto tied) {
    e = launch_plain(scan_step_kernel<decltype(t), decltype(v)::value, decltype(tau1)::value, decltype(tied)::value>, grid,
                     dim3(128), 0, st, p);
  });
  return e;
}

}  // namespace msgla
