// Element types of the operators around the attention call (rotary, layer
// norm, dropout): loads to fp32, stores rounded to nearest even, and the
// host-side choice of a kernel instantiation by type code.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"

namespace attn {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Element i of an array whose type is known at run time (weights and their
// gradients: one branch per element, the same for every thread).
__device__ __forceinline__ float load_as(const void* p, long long i, int dtype) {
  if (dtype == ATTN_FP32) return static_cast<const float*>(p)[i];
  if (dtype == ATTN_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_as(void* p, long long i, int dtype, float v) {
  if (dtype == ATTN_FP32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == ATTN_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else
    static_cast<__half*>(p)[i] = from_f32<__half>(v);
}

inline bool known_dtype(int dtype) {
  return dtype == ATTN_BF16 || dtype == ATTN_FP16 || dtype == ATTN_FP32;
}

// f(T{}) for the element type of a known code.
template <typename F>
inline int with_dtype(int dtype, F f) {
  if (dtype == ATTN_BF16) return f(__nv_bfloat16{});
  if (dtype == ATTN_FP16) return f(__half{});
  return f(float{});
}

}  // namespace attn
