// What the dense serving kernels (rope.cu, paged.cu) share: element
// conversions, dependent-launch helpers and the checks of a paged cache.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "hhr.h"

namespace hhr {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int type_size(int type) {
  switch (type) {
    case HHR_TYPE_BF16:
    case HHR_TYPE_F16: return 2;
    case HHR_TYPE_F32: return 4;
    case HHR_TYPE_E4M3: return 1;
    default: return 0;
  }
}

// Checks of a paged cache shared by every call that takes one.
inline int32_t check_paged(const hhr_paged* c) {
  if (!c) return HHR_ERR_INVALID_ARG;
  if (c->Hq < 1 || c->Hkv < 1 || c->d < 1 || c->page < 1 || c->n_pages < 1 || c->table_cols < 1)
    return HHR_ERR_INVALID_ARG;
  if (c->Hq % c->Hkv != 0 || c->reserved != 0) return HHR_ERR_INVALID_ARG;
  if (c->table_stride < c->table_cols) return HHR_ERR_INVALID_ARG;
  if (c->q_type != HHR_TYPE_BF16 && c->q_type != HHR_TYPE_F16) return HHR_ERR_INVALID_ARG;
  if (c->kv_type != c->q_type && c->kv_type != HHR_TYPE_E4M3) return HHR_ERR_INVALID_ARG;
  if (c->kv_type == HHR_TYPE_E4M3) {
    if (!(c->k_scale > 0) || !(c->v_scale > 0) || !std::isfinite(c->k_scale) || !std::isfinite(c->v_scale) ||
        !std::isfinite(1.0f / c->k_scale) || !std::isfinite(1.0f / c->v_scale))
      return HHR_ERR_INVALID_ARG;
  } else if (c->k_scale != 1.0f || c->v_scale != 1.0f) {
    return HHR_ERR_INVALID_ARG;
  }
  const int64_t unit = 16 / type_size(c->kv_type);
  const int64_t strides[6] = {c->k_page, c->k_head, c->k_tok, c->v_page, c->v_head, c->v_tok};
  for (int64_t s : strides)
    if (s < 1 || s % unit != 0) return HHR_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return HHR_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->Hq) * c->d >= (int64_t{1} << 31)) return HHR_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->table_cols) * c->page > (int64_t{1} << 31) - 64) return   // a tile's rows behind the last one have numbers too
    HHR_ERR_UNSUPPORTED;
  return HHR_OK;
}

// Programmatic dependent launch: the kernel may become resident while its
// predecessor on the stream finishes and waits for it before touching memory.
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename Args>
inline cudaError_t launch_dependent(void (*kern)(const Args), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_fp8_e4m3 x) { return static_cast<float>(x); }

// One rounding to nearest even; e4m3 saturates at its largest finite value.
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_fp8_e4m3 from_f32<__nv_fp8_e4m3>(float x) { return __nv_fp8_e4m3(x); }

// V consecutive elements, moved as one access where they fill a power of two
// of bytes up to 16.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

}  // namespace hhr
