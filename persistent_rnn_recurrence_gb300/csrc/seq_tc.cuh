// seq_tc.cuh -- device helpers of the sequence operators' tensor-core kernels: operand descriptors, fences between
// threads, copies and matrix products, tensor memory in rows of 16 columns, and values as sums of 16-bit parts.
#pragma once

#include <cstdint>
#include <type_traits>

#include "seq_common.cuh"

namespace prnn {
namespace tc {

// MN-major operand in 128-byte-swizzled tiles: 64 values of the M or N axis side by side, 8 steps of K
// per 1024 bytes; the next 64 values are `lead` bytes on.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
constexpr uint32_t kAMn = 1u << 15, kBMn = 1u << 16;
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return std::is_same<T, __half>::value ? f16_idesc(M, N) : bf16_idesc(M, N);
}
// The value, made at this place: sums with it are not hoisted out of the loop over chunks (a register
// pair for each of some sixty products would be spilled).
__device__ __forceinline__ uint64_t here(uint64_t v) {
  asm volatile("" : "+l"(v));
  return v;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void to_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
}
// One arrival for the whole warp, after every lane's work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15},"
      " [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two values as a packed pair of T, and what the packing left over.
template <typename T>
__device__ __forceinline__ uint32_t take(float2& v) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __float22half2_rn(v);
    const float2 b = __half22float2(h);
    v = fma2(b, both(-1.f), v);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    v = fma2(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)), both(-1.f), v);
    return u;
  }
}
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t u) {
  if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  else
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
// Values 2 j and 2 j + 1 of what was read from tensor memory.
__device__ __forceinline__ float2 pair_at(const uint32_t (&r)[16], int j) {
  return make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}
}  // namespace tc
}  // namespace prnn
