// dropout.cu -- dropout with an optional residual, its mask drawn from a
// counter-based generator and never stored.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products
// and three-way XORs turn (counter, key) into four words.  One block gives the
// words of four consecutive values, so a value's word depends on its index alone
// and the backward pass draws the same mask.
#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

// What all blocks of one launch share, made by the host.  The round keys are the seed plus multiples
// of two constants.  With the counter (index, high, offset), high and offset the same for
// the whole launch, one of the two products of round 0 and one of round 1 are the same for all threads
// too: 18 products are left of 20, and the 32 x 32 -> 64 bit product's rate is what bounds
// the generator.
struct Shared {
  uint32_t k[10][2];
  uint32_t c0_1;           // round 0: the first word it leaves
  uint32_t lo_1;           // its second word, the other product's low half
  uint32_t c3_0;           // offset's high word
  uint32_t hi_2, lo_2;     // round 1: the product of c0_1
};

constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u;

__device__ __forceinline__ uint4 philox(uint32_t index, const Shared& k) {
  // round 0 of (index, high, offset)
  uint64_t p0 = (uint64_t)index * kM0;
  uint32_t c2 = (uint32_t)(p0 >> 32) ^ k.c3_0 ^ k.k[0][1];
  uint32_t c3 = (uint32_t)p0;
  // round 1 of (c0_1, lo_1, c2, c3)
  uint64_t p1 = (uint64_t)c2 * kM1;
  uint32_t c0 = (uint32_t)(p1 >> 32) ^ k.lo_1 ^ k.k[1][0], c1 = (uint32_t)p1;
  c2 = k.hi_2 ^ c3 ^ k.k[1][1];
  c3 = k.lo_2;
#pragma unroll
  for (int i = 2; i < 10; ++i) {
    p0 = (uint64_t)c0 * kM0;
    p1 = (uint64_t)c2 * kM1;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k.k[i][0];
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k.k[i][1];
    c3 = (uint32_t)p0;
  }
  return make_uint4(c0, c1, c2, c3);
}

Shared shared_of(uint64_t seed, uint64_t offset, uint32_t high) {
  Shared s;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int i = 0; i < 10; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    s.k[i][0] = k0;
    s.k[i][1] = k1;
  }
  const uint64_t p1 = (uint64_t)(uint32_t)offset * kM1;
  s.c0_1 = (uint32_t)(p1 >> 32) ^ high ^ s.k[0][0];
  s.lo_1 = (uint32_t)p1;
  s.c3_0 = (uint32_t)(offset >> 32);
  const uint64_t p0 = (uint64_t)s.c0_1 * kM0;
  s.hi_2 = (uint32_t)(p0 >> 32);
  s.lo_2 = (uint32_t)p0;
  return s;
}

// V consecutive values per thread: 32 or 16 bytes of each tensor where all of them start on as many,
// else 4 values (one generator block) by single accesses.  The loads are issued before the generator
// runs.  What bounds it: bytes with fp32 data or a residual, the generator's products else.  8192 x
// 5760: bf16 with residual 42 us (all of the measured copy rate), bf16 alone 36 (0.79 of it), fp32 81
// and 56.  Five blocks an SM matter more than anything done by hand: the same kernel with the next
// pass's loads held in registers (93 of them, two blocks) took 62, with half the bytes per thread 68.
template <typename T, int V, bool VEC, bool RES>
__global__ void __launch_bounds__(256, 5) dropout_kernel(const __grid_constant__ DropoutArgs a,
                                                      const __grid_constant__ Shared key) {
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* y = static_cast<T*>(a.y);
  const float2 scale = both(a.scale);
  auto fetch = [&](long long at, Pack<T, V>& px, Pack<T, V>& pr) {
    if (VEC && at + V <= a.n) {
      px = load_once<T, V>(x + at);
      if (RES) pr = load_once<T, V>(res + at);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        px.v[j] = at + j < a.n ? x[at + j] : from_f32<T>(0.f);
        if (RES) pr.v[j] = at + j < a.n ? res[at + j] : from_f32<T>(0.f);
      }
    }
  };
  const long long at = (blockIdx.x * 256LL + threadIdx.x) * V;
  if (at < a.n) {
    Pack<T, V> px, pr;
    fetch(at, px, pr);
    uint32_t word[V];
#pragma unroll
    for (int b = 0; b < V / 4; ++b) {
      const uint4 w = philox((uint32_t)((uint64_t)at / 4) + b, key);
      word[4 * b] = w.x;
      word[4 * b + 1] = w.y;
      word[4 * b + 2] = w.z;
      word[4 * b + 3] = w.w;
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      float2 v = pair_of<T, V>(px, j);
      v.x = word[2 * j] >= a.limit ? v.x : 0.f;
      v.y = word[2 * j + 1] >= a.limit ? v.y : 0.f;
      v = RES ? fma2(v, scale, pair_of<T, V>(pr, j)) : mul2(v, scale);
      set_pair<T, V>(px, j, v);
    }
    if (VEC && at + V <= a.n) {
      store_pack<T, V>(y + at, px);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at + j < a.n) y[at + j] = px.v[j];
    }
  }
}

// One launch for every 2^34 values: the high word of the block index is a launch's own.
template <typename T, int V, bool VEC>
cudaError_t launch(DropoutArgs a, cudaStream_t s) {
  const long long n = a.n;
  for (long long from = 0, high = 0; from < n; from += 1LL << 34, ++high) {
    a.n = n - from < (1LL << 34) ? n - from : 1LL << 34;
    const long long want = ((a.n + V - 1) / V + 255) / 256;
    const int blocks = (int)want;  // at most 2^24
    const Shared key = shared_of(a.seed, a.offset, (uint32_t)high);
    if (a.residual)
      dropout_kernel<T, V, VEC, true><<<blocks, 256, 0, s>>>(a, key);
    else
      dropout_kernel<T, V, VEC, false><<<blocks, 256, 0, s>>>(a, key);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    a.x = static_cast<const T*>(a.x) + a.n;
    if (a.residual) a.residual = static_cast<const T*>(a.residual) + a.n;
    a.y = static_cast<T*>(a.y) + a.n;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                         reinterpret_cast<uintptr_t>(a.residual);
  cudaError_t e = cudaSuccess;
  if ((bits & 31) == 0) {
    PRNN_BY_DTYPE(a.dtype, T, (e = launch<T, 32 / sizeof(T), true>(a, s)));
  } else if ((bits & 15) == 0) {
    PRNN_BY_DTYPE(a.dtype, T, (e = launch<T, 16 / sizeof(T), true>(a, s)));
  } else {
    PRNN_BY_DTYPE(a.dtype, T, (e = launch<T, 4, false>(a, s)));
  }
  return e;
}

}  // namespace prnn
