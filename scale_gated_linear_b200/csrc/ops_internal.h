// ops_internal.h -- parameter blocks and device helpers shared by the gated
// recurrence (k_scan.cu), group normalisation (k_norm.cu) and their C entry
// points (ops_abi.cu). Not part of the public interface.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace msgla {

// Records `fmt` as the calling thread's last error and returns `code`.
int set_error(int code, const char* fmt, ...);

// Rows of channels: element (b, l, c) at ptr[b * batch + l * row + c].
struct Rows {
  void* ptr;
  long long batch, row;
};

// ---------------------------------------------------------------- gated recurrence
int scan_saved_rows(int dtype);  // rows between two saved states

// The gate as its kernels use it (set by the launches): 1 / tau; far = tau / 2 and the logit
// where softplus(-z) is that; the polynomial of (e^{-S / tau} - 1) / S, both halves of every
// packed operand.
struct DecayParams {
  float inv_tau, far, far_logit;
  float2 expm1[6];
};

struct ScanParams {
  int dtype, B, L, D, tied;
  int cluster;          // blocks per channel tile (set by the launches)
  float inv_tau;
  DecayParams gate;
  Rows x, z, h, dh, dx, dz;
  const uint8_t* mask;  // [B, L] or null
  const float* h0;      // [B, D] or null (zeros)
  float* last;          // [B, D]
  float* saved;         // [B, ceil(L / rows), D] states before rows 0, rows, 2 rows, ...; or null
  const float* dlast;   // [B, D] or null
  float* dh0;           // [B, D] or null
};
cudaError_t launch_scan_forward(const ScanParams& p, cudaStream_t st);
cudaError_t launch_scan_backward(const ScanParams& p, cudaStream_t st);

struct StepParams {
  int dtype, B, D, tied;
  float inv_tau;
  DecayParams gate;
  const void *x, *z;
  void* h;
  long long x_row, z_row, h_row;
  const uint8_t* mask;  // [B] or null
  float* state;         // [B, D]
};
cudaError_t launch_scan_step(const StepParams& p, cudaStream_t st);

// ---------------------------------------------------------------- group normalisation
struct NormParams {
  int dtype, C, G, act, center;
  int sms;  // of the call's device: the plans, and with them the workspace, depend on it
  float eps;
  long long N, S;
  Rows x, gate, y, dy, dx, dgate;  // gate.ptr null: no gate
  const float *w, *b;              // [C] or null (ones, zeros)
  const uint8_t* mask;             // [N, S] or null
  float* stats;                    // [N, G, 2] mean and 1 / sqrt(var + eps); forward: may be null
  float *dw, *db;                  // [C] or null
  void* workspace;
};
size_t norm_workspace(const NormParams& p, bool backward);
cudaError_t launch_norm_forward(const NormParams& p, cudaStream_t st);
cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t st);

// Lets `kernel` use `bytes` of dynamic shared memory on the current device; asked of the driver once
// for each kernel (a template argument, so each has its own mark) and device.
template <auto kernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A launch whose own status is returned: cudaGetLastError() after it would also report what another call left.
template <typename... KArgs, typename... Args>
cudaError_t launch_plain(void (*kernel)(KArgs...), dim3 grid, dim3 block, int shared, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

// ---------------------------------------------------------------- element types
enum : int { kBF16 = 0, kF16 = 1, kF32 = 2 };
enum : int { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
// both halves of a + b (packed pairs as sm100_ptx.cuh makes them)
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace msgla
