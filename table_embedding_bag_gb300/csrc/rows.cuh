// Row elements of the expert-layer and gradient kernels: fp32, fp16 or bf16
// values moved in vectors and computed on in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tbe.h"

namespace tbe {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// The one rounding of a result to its type (nearest even).
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// V elements moved by one access (V * sizeof(T) is 16, or V = 1).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T v[V];
};

inline int dtype_bytes(int32_t dtype) {
  return dtype == TBE_DT_F32 ? 4 : dtype == TBE_DT_F16 || dtype == TBE_DT_BF16 ? 2 : 0;
}

inline bool aligned_to(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

}  // namespace tbe
