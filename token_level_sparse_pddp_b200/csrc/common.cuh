// Shared device/host helpers of libtlsp (not part of the public ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "tlsp.h"

namespace tlsp {

// ----------------------------------------------------------------- host side

extern std::atomic<int64_t> g_launch_count;
void set_last_cuda_error(cudaError_t e);

// Returns TLSP_ERR_CUDA (and records the error) if the last launch failed.
inline int check_launch() {
  g_launch_count.fetch_add(1, std::memory_order_relaxed);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return TLSP_ERR_CUDA;
  }
  return TLSP_OK;
}

#define TLSP_TRY(expr)              \
  do {                              \
    int _rc = (expr);               \
    if (_rc != TLSP_OK) return _rc; \
  } while (0)

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Multiprocessor count of the current device, looked up once per device.
int device_sm_count();
// Raises kernel `fn`'s dynamic shared memory limit to `bytes` on the current
// device; the attribute call is made once per (kernel, device, size).
int ensure_smem_limit(const void* fn, int bytes);

// ----------------------------------------------------------------- dependent launches

// Launches a kernel, in clusters of `cluster` CTAs, that may start while the kernel before
// it in the stream is still finishing (programmatic dependent launch): its launch and
// first instructions then cost no time of their own (1 to 2 us a kernel, back to back).
// Each block has to execute wait_for_previous() before it touches memory that kernels
// before may write or read (unless the one before lets it start only after its own wait,
// and they do not depend on each other), and one block before it exits, so that kernels
// complete in their order.
template <class... Params, class... Args>
int launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster,
                     cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attrs;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  const int rc = check_launch();
  if (e == cudaSuccess) return rc;
  set_last_cuda_error(e);
  return TLSP_ERR_CUDA;
}
// Until the kernel before has completed and its writes are visible.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the kernel behind start once every block of this one has said so.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ----------------------------------------------------------------- device side

// Device status word: the first error wins, later ones are dropped.
__device__ __forceinline__ void record_status(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Loads 8 consecutive elements starting at p (16-byte aligned for bf16,
// 32-byte for fp32) into fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* out) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = __bfloat1622float2(h[i]);
    out[2 * i] = f.x;
    out[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float* out) {
  float4 a = *reinterpret_cast<const float4*>(p);
  float4 b = *reinterpret_cast<const float4*>(p + 4);
  out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
  out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Order-preserving map of fp32 onto uint32 (a < b  <=>  key(a) < key(b)),
// with -0 mapped like +0 so the two compare equal.
__device__ __forceinline__ uint32_t float_order_key(float f) {
  uint32_t b = __float_as_uint(f);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

}  // namespace tlsp
