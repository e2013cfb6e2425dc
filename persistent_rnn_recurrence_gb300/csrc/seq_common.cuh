// seq_common.cuh -- device helpers of the sequence operators: conversion
// between the storage types and fp32, sums over warps and blocks, and bounded waits.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tc_common.cuh"

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

// V consecutive elements of T in one access of up to 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& x) {
  *reinterpret_cast<Pack<T, V>*>(p) = x;
}
// Streaming forms for data that is touched once (read-only path, evict first).
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_once(const T* p) {
  Pack<T, V> r;
  if constexpr (sizeof(T) * V == 32) {
    const uint4* u = reinterpret_cast<const uint4*>(p);
    const uint4 w[2] = {__ldcs(u), __ldcs(u + 1)};
    r = *reinterpret_cast<const Pack<T, V>*>(w);
  } else if constexpr (sizeof(T) * V == 16) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    r = *reinterpret_cast<const Pack<T, V>*>(&u);
  } else {
    r = load_pack<T, V>(p);
  }
  return r;
}

// Two fp32 values side by side: Blackwell's paired add, multiply and fused multiply-add do both
// lanes in one instruction, each rounded as the single form rounds it.
__device__ __forceinline__ uint64_t as_u64(float2 v) {
  return (uint64_t)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 as_f2(uint64_t u) {
  return make_float2(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Elements 2i and 2i + 1 of a pack (i = 0 and a zero for a pack of one).
template <typename T, int V>
__device__ __forceinline__ float2 pair_of(const Pack<T, V>& p, int i) {
  if constexpr (V == 1)
    return make_float2(to_f32(p.v[0]), 0.f);
  else if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(p.v)[i]);
  else if constexpr (sizeof(T) == 2)
    return __half22float2(reinterpret_cast<const __half2*>(p.v)[i]);
  else
    return make_float2(to_f32(p.v[2 * i]), to_f32(p.v[2 * i + 1]));
}
template <typename T, int V>
__device__ __forceinline__ void set_pair(Pack<T, V>& p, int i, float2 f) {
  if constexpr (V == 1)
    p.v[0] = from_f32<T>(f.x);
  else if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    reinterpret_cast<__nv_bfloat162*>(p.v)[i] = __float22bfloat162_rn(f);
  else if constexpr (sizeof(T) == 2)
    reinterpret_cast<__half2*>(p.v)[i] = __float22half2_rn(f);
  else {
    p.v[2 * i] = from_f32<T>(f.x);
    p.v[2 * i + 1] = from_f32<T>(f.y);
  }
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

// Waits of the sequence operators' kernels for their own copies and matrix products.  Each one ends
// once it has lasted this long by itself, however long its block has been at work; the word that
// prnn_sequence_status reports is then set.
constexpr uint64_t kSeqWaitNs = 2000ull * 1000 * 1000;

// Waits for the phase of `bar` with the given parity.  A wait that runs out clears `ok`; the thread goes on,
// and with `ok` cleared its later waits end after the first polls, so that the block comes to its end.
// The clock is read only where 256 polls have not been enough.
__device__ __forceinline__ void seq_wait(uint64_t* bar, uint32_t parity, bool& ok) {
  uint32_t polls = 0;
  uint64_t since = 0;
  while (!tc::mbar_try_wait(bar, parity)) {
    if ((++polls & 255u) != 0u) continue;
    const uint64_t now = global_ns();
    if (since == 0) since = now;
    if (!ok || now - since > kSeqWaitNs) {
      ok = false;
      return;
    }
  }
}

// Run `f.template operator()<T>()` with the element type of dtype.
#define PRNN_BY_DTYPE(dtype, T, ...)                 \
  switch (dtype) {                                   \
    case PRNN_F32: { using T = float; __VA_ARGS__; break; }          \
    case PRNN_F16: { using T = __half; __VA_ARGS__; break; }         \
    default: { using T = __nv_bfloat16; __VA_ARGS__; break; }        \
  }

}  // namespace prnn
