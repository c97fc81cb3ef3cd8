// ops_abi.cu -- C entry points of the gated recurrence and of group normalisation
// (include/msgla.h): argument checks, parameter blocks and launches. Nothing here
// throws: it allocates no memory and its containers have fixed sizes.
#include <cmath>
#include <cstring>

#include "../../include/msgla.h"
#include "ops_internal.h"

using namespace msgla;

namespace {

// Reported by this call, and so taken out of the thread's last error: no later call finds it there.
int cuda_error(cudaError_t e, const char* what) {
  cudaGetLastError();
  return set_error(MSGLA_ERR_CUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

// Makes `dev` the current device for a call, and the previous one again.
struct Device {
  int prev = -1;
  bool moved = false;
  cudaError_t e;
  explicit Device(int dev) {
    e = cudaGetDevice(&prev);
    if (e != cudaSuccess || prev == dev) return;
    e = cudaSetDevice(dev);
    moved = true;
  }
  ~Device() {
    if (moved) cudaSetDevice(prev);
  }
};

int esize(int dtype) { return dtype == MSGLA_F32 ? 4 : 2; }

// The spans of a call's buffers: an output may meet no other one, unless both are rows of the same strides
// that lie side by side (halves of one tensor).
struct Spans {
  static constexpr int kMax = 16;
  struct One {
    const char* name;
    uintptr_t lo, hi;
    bool out;
    long long B, L, batch, row, width;  // of rows, in bytes; width 0: no rows
  } a[kMax];
  int n = 0;
  void add(const char* name, const void* p, unsigned long long bytes, bool out) {
    if (!p || !bytes || n == kMax) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    a[n++] = {name, lo, lo + bytes, out, 0, 0, 0, 0, 0};
  }
  void add_rows(const char* name, const msgla_rows& r, long long B, long long L, long long C, int size, bool out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(r.data);
    const long long batch = r.batch_stride * size, row = r.row_stride * size, width = C * size;
    if (n == kMax) return;
    a[n++] = {name, lo, lo + ((B - 1) * batch + (L - 1) * row + width), out, B, L, batch, row, width};
  }
  // Whether a row of x and the row of y in its place lie in one slot of the inner stride, and all of those in one of
  // the outer stride; or all inner rows of x beside all of y in a slot of the outer stride.
  static bool side_by_side(const One& x, const One& y) {
    if (!x.width || x.width != y.width || x.B != y.B || x.L != y.L) return false;
    if ((x.B > 1 && x.batch != y.batch) || (x.L > 1 && x.row != y.row)) return false;
    const long long apart = x.lo < y.lo ? static_cast<long long>(y.lo - x.lo) : static_cast<long long>(x.lo - y.lo);
    const auto nested = [&](long long n_in, long long in, long long n_out, long long out) {
      const long long reach = (n_in - 1) * in + x.width;  // of the inner rows of one
      return (n_in <= 1 || apart + x.width <= in || apart >= reach) && (n_out <= 1 || apart + reach <= out);
    };
    return apart >= x.width && (nested(x.L, x.row, x.B, x.batch) || nested(x.B, x.batch, x.L, x.row));
  }
  int check() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((a[i].out || a[j].out) && a[i].lo < a[j].hi && a[j].lo < a[i].hi && !side_by_side(a[i], a[j]))
          return set_error(MSGLA_ERR_INVALID_ARG, "%s and %s overlap", a[j].name, a[i].name);
    return MSGLA_OK;
  }
};

// Checks rows [B, L, C] and adds their span; *out receives the kernel's form.
int take_rows(const char* name, const msgla_rows* r, long long B, long long L, long long C, int dtype, bool out,
              Spans& spans, Rows* to) {
  if (!r || !r->data) return set_error(MSGLA_ERR_INVALID_ARG, "%s is NULL", name);
  const long long sb = r->batch_stride, sl = r->row_stride, most = 1LL << 46;
  if (sb < 0 || sl < 0 || sb >= most || sl >= most)
    return set_error(MSGLA_ERR_INVALID_ARG, "%s: strides %lld, %lld outside [0, 2^46)", name, sb, sl);
  if (reinterpret_cast<uintptr_t>(r->data) % esize(dtype))
    return set_error(MSGLA_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  // the products stay below 2^63 in magnitude only as floating point: spans this long do not exist
  const double last = static_cast<double>(B - 1) * sb + static_cast<double>(L - 1) * sl + C;
  if (last > 1e15) return set_error(MSGLA_ERR_INVALID_ARG, "%s spans more than 10^15 elements", name);
  if (out) {  // one of the two strides steps over everything the other reaches
    const long long row_span = (L - 1) * sl + C, batch_span = (B - 1) * sb + C;
    const bool rows_inside = (L <= 1 || sl >= C) && (B <= 1 || sb >= row_span);
    const bool batches_inside = (B <= 1 || sb >= C) && (L <= 1 || sl >= batch_span);
    if (!rows_inside && !batches_inside)
      return set_error(MSGLA_ERR_INVALID_ARG, "%s: strides %lld, %lld make elements coincide", name, sb, sl);
  }
  spans.add_rows(name, *r, B, L, C, esize(dtype), out);
  *to = Rows{r->data, B <= 1 ? 0 : sb, L <= 1 ? 0 : sl};
  return MSGLA_OK;
}

int take_f32(const char* name, const float* p, bool needed) {
  if (!p) return needed ? set_error(MSGLA_ERR_INVALID_ARG, "%s is NULL", name) : MSGLA_OK;
  if (reinterpret_cast<uintptr_t>(p) % 4) return set_error(MSGLA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
  return MSGLA_OK;
}

#define TRY(expr)        \
  do {                   \
    const int st_ = (expr); \
    if (st_) return st_; \
  } while (0)

int check_scan(const msgla_scan_config* c, int B, int L) {
  if (!c) return set_error(MSGLA_ERR_INVALID_ARG, "cfg is NULL");
  if (c->dtype < MSGLA_BF16 || c->dtype > MSGLA_F32) return set_error(MSGLA_ERR_INVALID_ARG, "dtype=%d", c->dtype);
  if (c->D < 1 || c->D > 1 << 24) return set_error(MSGLA_ERR_INVALID_ARG, "D=%d outside [1, 2^24]", c->D);
  if (c->tied != 0 && c->tied != 1) return set_error(MSGLA_ERR_INVALID_ARG, "tied=%d must be 0 or 1", c->tied);
  if (!(c->gate_normalizer >= 0x1p-10f && c->gate_normalizer <= 0x1p20f))
    return set_error(MSGLA_ERR_INVALID_ARG, "gate_normalizer=%g outside [2^-10, 2^20]", c->gate_normalizer);
  if (B < 0 || B > 65535) return set_error(MSGLA_ERR_INVALID_ARG, "B=%d outside [0, 65535]", B);
  if (L < 0 || L > 1 << 30) return set_error(MSGLA_ERR_INVALID_ARG, "L=%d outside [0, 2^30]", L);
  return MSGLA_OK;
}

size_t saved_bytes(const msgla_scan_config* c, int B, int L) {
  const int rows = scan_saved_rows(c->dtype);
  return static_cast<size_t>(B) * ((static_cast<size_t>(L) + rows - 1) / rows) * c->D * 4;
}

ScanParams scan_params(const msgla_scan_config* c, int B, int L, const void* M) {
  ScanParams p = {};
  p.dtype = c->dtype;
  p.B = B;
  p.L = L;
  p.D = c->D;
  p.tied = c->tied;
  p.inv_tau = 1.f / c->gate_normalizer;
  p.mask = static_cast<const uint8_t*>(M);
  return p;
}

// dst[0 .. bytes) = src, or zeros
int copy_or_zero(void* dst, const void* src, size_t bytes, cudaStream_t st) {
  if (dst == src) return MSGLA_OK;
  const cudaError_t e = src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st)
                            : cudaMemsetAsync(dst, 0, bytes, st);
  return e == cudaSuccess ? MSGLA_OK : cuda_error(e, src ? "cudaMemcpyAsync" : "cudaMemsetAsync");
}

int check_norm(const msgla_norm_config* c, long long N, long long S) {
  if (!c) return set_error(MSGLA_ERR_INVALID_ARG, "cfg is NULL");
  if (c->dtype < MSGLA_BF16 || c->dtype > MSGLA_F32) return set_error(MSGLA_ERR_INVALID_ARG, "dtype=%d", c->dtype);
  if (c->C < 1 || c->C > 1 << 24) return set_error(MSGLA_ERR_INVALID_ARG, "C=%d outside [1, 2^24]", c->C);
  if (c->groups < 1 || c->C % c->groups)
    return set_error(MSGLA_ERR_INVALID_ARG, "groups=%d must divide C=%d", c->groups, c->C);
  if (c->activation < MSGLA_ACT_NONE || c->activation > MSGLA_ACT_SIGMOID)
    return set_error(MSGLA_ERR_INVALID_ARG, "activation=%d", c->activation);
  if (c->center != 0 && c->center != 1) return set_error(MSGLA_ERR_INVALID_ARG, "center=%d must be 0 or 1", c->center);
  if (!(c->eps > 0.f) || !std::isfinite(c->eps))
    return set_error(MSGLA_ERR_INVALID_ARG, "eps must be positive and finite");
  const long long most = 1LL << 31;
  if (N < 0 || S < 0 || N >= most || S >= most || N * c->groups >= most || N * S >= most)
    return set_error(MSGLA_ERR_INVALID_ARG, "N=%lld, S=%lld: N * groups and N * S must be in [0, 2^31)", N, S);
  return MSGLA_OK;
}

// The SMs of device `dev` (148 where no GPU can be asked, so that sizes can be made there).
int count_sms(int dev, int* sms) {
  const cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) return MSGLA_OK;
  if (e == cudaErrorInvalidDevice) return cuda_error(e, "asking for the device");
  *sms = 148;
  return MSGLA_OK;
}

int norm_params(const msgla_norm_config* c, long long N, long long S, NormParams* to) {
  NormParams p = {};
  p.dtype = c->dtype;
  p.C = c->C;
  p.G = c->groups;
  p.act = c->activation;
  p.center = c->center;
  p.eps = c->eps;
  p.N = N;
  p.S = S;
  *to = p;
  return count_sms(c->device, &to->sms);
}

int check_workspace(const NormParams& p, bool backward, void* ws, size_t bytes, Spans& spans) {
  const size_t need = norm_workspace(p, backward);
  if (!need) return MSGLA_OK;
  if (!ws || bytes < need)
    return set_error(MSGLA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? bytes : size_t(0), need);
  if (reinterpret_cast<uintptr_t>(ws) % 256) return set_error(MSGLA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  spans.add("workspace", ws, need, true);
  return MSGLA_OK;
}

#define ON_DEVICE(dev)       \
  Device guard(dev);         \
  if (guard.e != cudaSuccess) return cuda_error(guard.e, "cudaSetDevice")

}  // namespace

extern "C" {

int msgla_scan_saved_size(const msgla_scan_config* cfg, int B, int L, size_t* bytes) {
  TRY(check_scan(cfg, B, L));
  if (!bytes) return set_error(MSGLA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = saved_bytes(cfg, B, L);
  return MSGLA_OK;
}

int msgla_scan_forward(const msgla_scan_config* cfg, int B, int L, const msgla_rows* x, const msgla_rows* z,
                       const void* M, const float* h0, const msgla_rows* h, float* h_last, float* saved,
                       void* stream) {
  TRY(check_scan(cfg, B, L));
  if (B == 0) return MSGLA_OK;
  TRY(take_f32("h0", h0, false));
  TRY(take_f32("h_last", h_last, true));
  TRY(take_f32("saved", saved, false));
  const size_t states = static_cast<size_t>(B) * cfg->D * 4;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ScanParams p = scan_params(cfg, B, L, M);
  Spans spans;
  if (h0 != h_last) spans.add("h0", h0, states, false);
  spans.add("h_last", h_last, states, true);
  if (L > 0) {
    TRY(take_rows("x", x, B, L, cfg->D, cfg->dtype, false, spans, &p.x));
    TRY(take_rows("z", z, B, L, cfg->D, cfg->dtype, false, spans, &p.z));
    TRY(take_rows("h", h, B, L, cfg->D, cfg->dtype, true, spans, &p.h));
    spans.add("M", M, static_cast<size_t>(B) * L, false);
    spans.add("saved", saved, saved_bytes(cfg, B, L), true);
  }
  TRY(spans.check());
  ON_DEVICE(cfg->device);
  if (L == 0) return copy_or_zero(h_last, h0, states, st);
  p.h0 = h0;
  p.last = h_last;
  p.saved = saved;
  const cudaError_t e = launch_scan_forward(p, st);
  return e == cudaSuccess ? MSGLA_OK : cuda_error(e, "the recurrence's launch");
}

int msgla_scan_backward(const msgla_scan_config* cfg, int B, int L, const msgla_rows* x, const msgla_rows* z,
                        const void* M, const float* saved, const msgla_rows* dh, const float* dh_last,
                        const msgla_rows* dx, const msgla_rows* dz, float* dh0, void* stream) {
  TRY(check_scan(cfg, B, L));
  if (B == 0) return MSGLA_OK;
  TRY(take_f32("dh_last", dh_last, false));
  TRY(take_f32("dh0", dh0, false));
  TRY(take_f32("saved", saved, L > 0));
  const size_t states = static_cast<size_t>(B) * cfg->D * 4;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ScanParams p = scan_params(cfg, B, L, M);
  Spans spans;
  if (dh0 != dh_last) spans.add("dh_last", dh_last, states, false);
  spans.add("dh0", dh0, states, true);
  if (L > 0) {
    TRY(take_rows("x", x, B, L, cfg->D, cfg->dtype, false, spans, &p.x));
    TRY(take_rows("z", z, B, L, cfg->D, cfg->dtype, false, spans, &p.z));
    if (dh && dh->data) TRY(take_rows("dh", dh, B, L, cfg->D, cfg->dtype, false, spans, &p.dh));
    TRY(take_rows("dx", dx, B, L, cfg->D, cfg->dtype, true, spans, &p.dx));
    TRY(take_rows("dz", dz, B, L, cfg->D, cfg->dtype, true, spans, &p.dz));
    spans.add("M", M, static_cast<size_t>(B) * L, false);
    spans.add("saved", saved, saved_bytes(cfg, B, L), false);
  }
  TRY(spans.check());
  ON_DEVICE(cfg->device);
  if (L == 0) return dh0 ? copy_or_zero(dh0, dh_last, states, st) : MSGLA_OK;
  p.saved = const_cast<float*>(saved);
  p.dlast = dh_last;
  p.dh0 = dh0;
  const cudaError_t e = launch_scan_backward(p, st);
  return e == cudaSuccess ? MSGLA_OK : cuda_error(e, "the recurrence's gradient launch");
}

int msgla_scan_step(const msgla_scan_config* cfg, int B, const msgla_rows* x, const msgla_rows* z, const void* M,
                    float* state, const msgla_rows* h, void* stream) {
  TRY(check_scan(cfg, B, 1));
  if (B == 0) return MSGLA_OK;
  TRY(take_f32("state", state, true));
  Spans spans;
  Rows rx, rz, rh;
  TRY(take_rows("x", x, B, 1, cfg->D, cfg->dtype, false, spans, &rx));
  TRY(take_rows("z", z, B, 1, cfg->D, cfg->dtype, false, spans, &rz));
  TRY(take_rows("h", h, B, 1, cfg->D, cfg->dtype, true, spans, &rh));
  spans.add("M", M, B, false);
  spans.add("state", state, static_cast<size_t>(B) * cfg->D * 4, true);
  TRY(spans.check());
  ON_DEVICE(cfg->device);
  StepParams p = {};
  p.dtype = cfg->dtype;
  p.B = B;
  p.D = cfg->D;
  p.tied = cfg->tied;
  p.inv_tau = 1.f / cfg->gate_normalizer;
  p.x = rx.ptr;
  p.z = rz.ptr;
  p.h = rh.ptr;
  p.x_row = rx.batch;
  p.z_row = rz.batch;
  p.h_row = rh.batch;
  p.mask = static_cast<const uint8_t*>(M);
  p.state = state;
  const cudaError_t e = launch_scan_step(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MSGLA_OK : cuda_error(e, "the recurrence step's launch");
}

int msgla_group_norm_workspace_size(const msgla_norm_config* cfg, long long N, long long S, int gradients,
                                    size_t* bytes) {
  TRY(check_norm(cfg, N, S));
  if (!bytes) return set_error(MSGLA_ERR_INVALID_ARG, "bytes is NULL");
  NormParams p;
  TRY(norm_params(cfg, N, S, &p));
  *bytes = N * S == 0 ? 0 : norm_workspace(p, gradients != 0);
  return MSGLA_OK;
}

int msgla_group_norm_forward(const msgla_norm_config* cfg, long long N, long long S, const msgla_rows* x,
                             const msgla_rows* gate, const float* weight, const float* bias, const void* M,
                             const msgla_rows* y, float* stats, void* workspace, size_t workspace_bytes,
                             void* stream) {
  TRY(check_norm(cfg, N, S));
  if (N * S == 0) return MSGLA_OK;
  TRY(take_f32("weight", weight, false));
  TRY(take_f32("bias", bias, false));
  if (reinterpret_cast<uintptr_t>(stats) % 8) return set_error(MSGLA_ERR_INVALID_ARG, "stats is not 8-byte aligned");
  NormParams p;
  TRY(norm_params(cfg, N, S, &p));
  Spans spans;
  TRY(take_rows("x", x, N, S, cfg->C, cfg->dtype, false, spans, &p.x));
  if (gate) TRY(take_rows("gate", gate, N, S, cfg->C, cfg->dtype, false, spans, &p.gate));
  TRY(take_rows("y", y, N, S, cfg->C, cfg->dtype, true, spans, &p.y));
  spans.add("weight", weight, cfg->C * 4ull, false);
  spans.add("bias", bias, cfg->C * 4ull, false);
  spans.add("M", M, static_cast<size_t>(N) * S, false);
  spans.add("stats", stats, static_cast<size_t>(N) * cfg->groups * 8, true);
  TRY(check_workspace(p, false, workspace, workspace_bytes, spans));
  TRY(spans.check());
  ON_DEVICE(cfg->device);
  p.w = weight;
  p.b = bias;
  p.mask = static_cast<const uint8_t*>(M);
  p.stats = stats;
  p.workspace = workspace;
  const cudaError_t e = launch_norm_forward(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MSGLA_OK : cuda_error(e, "the normalisation's launch");
}

int msgla_group_norm_backward(const msgla_norm_config* cfg, long long N, long long S, const msgla_rows* x,
                              const msgla_rows* gate, const float* weight, const float* bias, const void* M,
                              const float* stats, const msgla_rows* dy, const msgla_rows* dx,
                              const msgla_rows* dgate, float* dweight, float* dbias, void* workspace,
                              size_t workspace_bytes, void* stream) {
  TRY(check_norm(cfg, N, S));
  TRY(take_f32("weight", weight, false));
  TRY(take_f32("bias", bias, false));
  TRY(take_f32("dweight", dweight, false));
  TRY(take_f32("dbias", dbias, false));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N * S == 0) {
    ON_DEVICE(cfg->device);
    if (dweight) TRY(copy_or_zero(dweight, nullptr, cfg->C * 4ull, st));
    return dbias ? copy_or_zero(dbias, nullptr, cfg->C * 4ull, st) : MSGLA_OK;
  }
  if (!stats || reinterpret_cast<uintptr_t>(stats) % 8)
    return set_error(MSGLA_ERR_INVALID_ARG, "stats is NULL or not 8-byte aligned");
  if (!gate != !dgate) return set_error(MSGLA_ERR_INVALID_ARG, "gate and dgate go together");
  NormParams p;
  TRY(norm_params(cfg, N, S, &p));
  Spans spans;
  TRY(take_rows("x", x, N, S, cfg->C, cfg->dtype, false, spans, &p.x));
  if (gate) TRY(take_rows("gate", gate, N, S, cfg->C, cfg->dtype, false, spans, &p.gate));
  TRY(take_rows("dy", dy, N, S, cfg->C, cfg->dtype, false, spans, &p.dy));
  TRY(take_rows("dx", dx, N, S, cfg->C, cfg->dtype, true, spans, &p.dx));
  if (dgate) TRY(take_rows("dgate", dgate, N, S, cfg->C, cfg->dtype, true, spans, &p.dgate));
  spans.add("weight", weight, cfg->C * 4ull, false);
  spans.add("bias", bias, cfg->C * 4ull, false);
  spans.add("M", M, static_cast<size_t>(N) * S, false);
  spans.add("stats", stats, static_cast<size_t>(N) * cfg->groups * 8, false);
  spans.add("dweight", dweight, cfg->C * 4ull, true);
  spans.add("dbias", dbias, cfg->C * 4ull, true);
  TRY(check_workspace(p, true, workspace, workspace_bytes, spans));
  TRY(spans.check());
  ON_DEVICE(cfg->device);
  p.w = weight;
  p.b = bias;
  p.mask = static_cast<const uint8_t*>(M);
  p.stats = const_cast<float*>(stats);
  p.dw = dweight;
  p.db = dbias;
  p.workspace = workspace;
  const cudaError_t e = launch_norm_backward(p, st);
  return e == cudaSuccess ? MSGLA_OK : cuda_error(e, "the normalisation's gradient launch");
}

}  // extern "C"
