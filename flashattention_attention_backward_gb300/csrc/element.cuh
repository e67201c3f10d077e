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

// 16 bytes of T in registers, and their elements in fp32.
template <typename T>
struct Vec {
  static constexpr int kElems = 16 / sizeof(T);
  uint4 w;
};

__device__ __forceinline__ void unpack(const Vec<float>& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.w.x);
  f[1] = __uint_as_float(v.w.y);
  f[2] = __uint_as_float(v.w.z);
  f[3] = __uint_as_float(v.w.w);
}
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16>& v, float (&f)[8]) {
  const uint32_t w[4] = {v.w.x, v.w.y, v.w.z, v.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Vec<__half>& v, float (&f)[8]) {
  const uint32_t w[4] = {v.w.x, v.w.y, v.w.z, v.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ void pack(const float (&f)[4], Vec<float>& v) {
  v.w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec<__nv_bfloat16>& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  v.w = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec<__half>& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  v.w = make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
  Vec<T> v;
  v.w = *reinterpret_cast<const uint4*>(p);
  return v;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v) {
  *reinterpret_cast<uint4*>(p) = v.w;
}

inline bool known_dtype(int dtype) {
  return dtype == ATTN_BF16 || dtype == ATTN_FP16 || dtype == ATTN_FP32;
}

// Launches a kernel that begins with ptx::grid_dependency_wait(), so that its
// launch (not its work) overlaps the end of the stream's kernel before it: 0.3 to
// 0.5 us less a call in a graph (finalize of 1 x 2 x 256 x 64 1.7, not 1.9), up to
// 1.8 less for the layer norm backward called back to back (64 x 512: 6.3, not
// 8.1). `cluster`: blocks of a cluster, 0 for none.
template <typename... Params, typename... Args>
inline int launch_overlapped(void (*kern)(Params...), dim3 grid, int block, int smem, int cluster,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(static_cast<unsigned>(block));
  config.dynamicSmemBytes = static_cast<size_t>(smem);
  config.stream = stream;
  config.attrs = attrs;
  config.numAttrs = cluster > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&config, kern, args...) != cudaSuccess) {
    cudaGetLastError();  // reported here, not by a later call
    return ATTN_ERR_LAUNCH;
  }
  return ATTN_OK;
}

// f(T{}) for the element type of a known code.
template <typename F>
inline int with_dtype(int dtype, F f) {
  if (dtype == ATTN_BF16) return f(__nv_bfloat16{});
  if (dtype == ATTN_FP16) return f(__half{});
  return f(float{});
}

}  // namespace attn
