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

__device__ __forceinline__ uint4 philox(uint64_t index, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutArgs a) {
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* y = static_cast<T*>(a.y);
  const long long quads = (a.n + 3) / 4;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < quads;
       i += (long long)gridDim.x * blockDim.x) {
    const uint4 w = philox((uint64_t)i, a.offset, a.seed);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long at = 4 * i + j;
      if (at >= a.n) break;
      float v = word[j] >= a.limit ? to_f32(x[at]) * a.scale : 0.f;
      if (res) v += to_f32(res[at]);
      y[at] = from_f32<T>(v);
    }
  }
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  const long long want = ((a.n + 3) / 4 + 255) / 256;
  const int blocks = (int)(want < 152 * 32 ? want : 152 * 32);
  PRNN_BY_DTYPE(a.dtype, T, (dropout_kernel<T><<<blocks, 256, 0, s>>>(a)));
  return cudaGetLastError();
}

}  // namespace prnn
