// linear_attention_step.cu -- one token of linear attention with a decay per
// head: S <- l S + k v^T, o = scale S^T q, the fp32 state in place.
//
// Bound by memory: the state is read and written once, 8 dk dv bytes per head
// against 5 dk dv flops.
#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

// One block per (sequence, head), 32 columns of the state per warp row.
template <typename T>
__global__ void __launch_bounds__(256) la_step_kernel(LaStepArgs a) {
  __shared__ float qs[256], ks[256], part[8][33];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T* o = static_cast<T*>(a.o) + b * a.ob + h * a.oh;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    for (int c = threadIdx.x; c < a.dv; c += 256) o[c] = from_f32<T>(0.f);
    return;
  }
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + (h / a.q.share) * a.q.sh;
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + (h / a.k.share) * a.k.sh;
  const T* v = static_cast<const T*>(a.v.p) + b * a.v.sb + (h / a.v.share) * a.v.sh;
  float* S = a.state + ((size_t)slot * a.H + h) * a.dk * a.dv;
  for (int i = threadIdx.x; i < a.dk; i += 256) {
    qs[i] = to_f32(q[i]);
    ks[i] = to_f32(k[i]);
  }
  const float l = expf(a.log_decay[h]);
  __syncthreads();
  for (int c0 = 0; c0 < a.dv; c0 += 32) {
    const int c = c0 + lane;
    float s = 0.f;
    if (c < a.dv) {
      const float vc = to_f32(v[c]);
      for (int i = warp; i < a.dk; i += 8) {
        const float n = l * S[(size_t)i * a.dv + c] + ks[i] * vc;
        S[(size_t)i * a.dv + c] = n;
        s = fmaf(qs[i], n, s);
      }
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.dv) {
      s = 0.f;
      for (int w = 0; w < 8; ++w) s += part[w][lane];
      o[c] = from_f32<T>(a.scale * s);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_la_step(const LaStepArgs& a, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  PRNN_BY_DTYPE(a.dtype, T, (la_step_kernel<T><<<a.B * a.H, 256, 0, s>>>(a)));
  return cudaGetLastError();
}

}  // namespace prnn
