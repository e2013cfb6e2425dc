// linear_attention_step.cu -- one token of linear attention with a decay per
// head: S <- l S + k v^T, o = scale S^T q, the fp32 state in place.
//
// Bound by memory: the state is read and written once, 8 dk dv bytes per head against 5 dk dv flops.
// Measured on GB300: 96 sequences of 16 heads of 128 x 128 36.6 us (0.82 of the copy rate of 6.69
// TB/s), 16 of them 10.5, one of 8 heads of 64 x 64 2.5 (a launch).
#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

constexpr int kThreads = 256, kInFlight = 8;

// One block: one (sequence, head) and `slice` columns of its state.  TX threads side by side hold
// V columns each and the 256 / TX rows of threads share the dk rows; every thread keeps kInFlight
// loads of the state in flight, the first of them issued before q, k and v arrive.
template <typename T, int V, int TX>
__global__ void __launch_bounds__(kThreads) la_step_kernel(LaStepArgs a, int slice) {
  constexpr int TY = kThreads / TX;
  __shared__ float qs[256], ks[256], part[TY][TX * V + 1];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int c0 = blockIdx.y * slice, c = c0 + tx * V;
  const int ncol = min(slice, a.dv - c0);
  T* o = static_cast<T*>(a.o) + b * a.ob + h * a.oh + c0;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    for (int i = threadIdx.x; i < ncol; i += kThreads) o[i] = from_f32<T>(0.f);
    return;
  }
  float* S = a.state + ((size_t)slot * a.H + h) * a.dk * a.dv + c;
  const bool mine = tx * V < ncol;  // V divides dv and slice: all V columns or none
  Pack<float, V> st[kInFlight];
#pragma unroll
  for (int u = 0; u < kInFlight; ++u) {
    const int i = ty + u * TY;
    if (mine && i < a.dk) st[u] = load_pack<float, V>(S + (size_t)i * a.dv);
  }
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + (h / a.q.share) * a.q.sh;
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + (h / a.k.share) * a.k.sh;
  const T* v = static_cast<const T*>(a.v.p) + b * a.v.sb + (h / a.v.share) * a.v.sh;
  for (int i = threadIdx.x; i < a.dk; i += kThreads) {
    qs[i] = to_f32(q[i]);
    ks[i] = to_f32(k[i]);
  }
  const float l = expf(a.log_decay[h]);
  float vc[V], sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    vc[j] = mine ? to_f32(v[c + j]) : 0.f;
    sum[j] = 0.f;
  }
  __syncthreads();
  for (int i0 = ty; i0 < a.dk; i0 += kInFlight * TY) {
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int i = i0 + u * TY;
      if (!mine || i >= a.dk) continue;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        st[u].v[j] = fmaf(l, st[u].v[j], ks[i] * vc[j]);
        sum[j] = fmaf(qs[i], st[u].v[j], sum[j]);
      }
      store_pack<float, V>(S + (size_t)i * a.dv, st[u]);
      const int next = i + kInFlight * TY;
      if (next < a.dk) st[u] = load_pack<float, V>(S + (size_t)next * a.dv);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) part[ty][tx * V + j] = sum[j];
  __syncthreads();
  for (int i = threadIdx.x; i < ncol; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < TY; ++w) s += part[w][i];
    o[i] = from_f32<T>(a.scale * s);
  }
}

template <typename T, int V>
void launch(const LaStepArgs& a, int slice, cudaStream_t s) {
  const dim3 grid(a.B * a.H, (a.dv + slice - 1) / slice);
  const int tx = (slice + V - 1) / V;
  if (tx <= 4)
    la_step_kernel<T, V, 4><<<grid, kThreads, 0, s>>>(a, slice);
  else if (tx <= 8)
    la_step_kernel<T, V, 8><<<grid, kThreads, 0, s>>>(a, slice);
  else if (tx <= 16)
    la_step_kernel<T, V, 16><<<grid, kThreads, 0, s>>>(a, slice);
  else
    la_step_kernel<T, V, 32><<<grid, kThreads, 0, s>>>(a, slice);
}

}  // namespace

cudaError_t launch_la_step(const LaStepArgs& a, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  const bool vec = a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  // Columns per block: up to 32 threads' worth, narrower while the blocks are too few to fill the SMs.
  int slice = vec ? 128 : 32;
  while (slice > a.dv && slice > 16) slice /= 2;
  if (slice < a.dv && slice * 2 >= a.dv && slice < (vec ? 128 : 32)) slice *= 2;
  while (slice > 16 && (long long)a.B * a.H * ((a.dv + slice - 1) / slice) < seq_sm_count()) slice /= 2;
  if (vec) {
    PRNN_BY_DTYPE(a.dtype, T, (launch<T, 4>(a, slice, s)));
  } else {
    PRNN_BY_DTYPE(a.dtype, T, (launch<T, 1>(a, slice, s)));
  }
  return cudaGetLastError();
}

}  // namespace prnn
