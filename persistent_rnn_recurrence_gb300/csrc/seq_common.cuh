// seq_common.cuh -- device helpers of the sequence operators: conversion
// between the storage types and fp32, and sums over warps and blocks.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace prnn {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over a block of whole warps; `part` holds one float per warp.  Every
// thread gets the sum, added in the same order.  part may be reused after the next barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = warp_sum(v);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps; ++w) s += part[w];
  return s;
}

// decay^n for log-decay ld and n >= 0, with decay^0 = 1 even for decay = 0.
__device__ __forceinline__ float decay_pow(float ld, int n) {
  return n == 0 ? 1.f : expf(ld * (float)n);
}

// Run `f.template operator()<T>()` with the element type of dtype.
#define PRNN_BY_DTYPE(dtype, T, ...)                 \
  switch (dtype) {                                   \
    case PRNN_F32: { using T = float; __VA_ARGS__; break; }          \
    case PRNN_F16: { using T = __half; __VA_ARGS__; break; }         \
    default: { using T = __nv_bfloat16; __VA_ARGS__; break; }        \
  }

}  // namespace prnn
