// gated_delta_step.cu -- one token of the gated delta rule: S' = a S, e = v - S'^T k, S <- S' + k (beta e)^T,
// o = scale S^T q, the fp32 state in place.
//
// Bound by memory: the state is read and written once, 8 dk dv bytes per head against 7 dk dv flops.  A block holds
// all dk rows of 32 columns in registers, so that the state is read once although its product with k comes before
// its update; S^T q = S'^T q + (k . q) beta e, so both products with S' are summed at once and one
// exchange serves both.  Measured on GB300: 96 sequences of 16 heads of 128 x 128 36.9 us (0.80 of the copy rate of
// 6.78 TB/s), one of 8 heads of 64 x 64 3.7 (a launch).
#include <algorithm>

#include "gated_delta.h"
#include "seq_common.cuh"

namespace prnn {
namespace {

constexpr int kThreads = 256, kSlice = 32;

// TX threads side by side hold V columns each (TX V = 32), the 256 / TX rows of threads R rows each.
template <typename T, int V, int R>
__global__ void __launch_bounds__(kThreads) gd_step_kernel(const __grid_constant__ GdStepArgs a) {
  constexpr int TX = kSlice / V, TY = kThreads / TX;
  __shared__ float qs[256], ks[256], sums[2][TY][kSlice + 1], out[2][kSlice], kq_part[kThreads / 32];
  const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, c0 = blockIdx.y * kSlice, c = c0 + tx * V;
  const int ncol = min(kSlice, a.dv - c0);
  T* o = static_cast<T*>(a.o) + b * a.ob + h * a.oh + c0;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    if (tid < ncol) o[tid] = from_f32<T>(0.f);
    return;
  }
  float* S = a.state + ((size_t)slot * a.H + h) * a.dk * a.dv + c;
  const bool mine = tx * V < ncol;  // V divides dv: all V columns or none
  Pack<float, V> st[R];
#pragma unroll
  for (int u = 0; u < R; ++u) {
    const int i = ty + u * TY;
    if (mine && i < a.dk) {
      st[u] = load_pack<float, V>(S + (size_t)i * a.dv);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) st[u].v[j] = 0.f;
    }
  }
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + (h / a.q.share) * a.q.sh;
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + (h / a.k.share) * a.k.sh;
  const T* v = static_cast<const T*>(a.v.p) + b * a.v.sb + h * a.v.sh;
  float kq = 0.f;
  if (tid < a.dk) {  // dk <= 256
    qs[tid] = to_f32(q[tid]);
    ks[tid] = to_f32(k[tid]);
    kq = qs[tid] * ks[tid];
  }
  const float decay = expf(a.g[b * a.gb + h * a.gh]), beta = a.beta[b * a.bb + h * a.bh];
  const float value = tid < ncol ? to_f32(v[c0 + tid]) : 0.f;
  kq = warp_sum(kq);
  if ((tid & 31) == 0) kq_part[tid >> 5] = kq;
  __syncthreads();
  float sk[V], sq[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sk[j] = sq[j] = 0.f;
#pragma unroll
  for (int u = 0; u < R; ++u) {
    const int i = ty + u * TY;
    const float ki = i < a.dk ? ks[i] : 0.f, qi = i < a.dk ? qs[i] : 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      st[u].v[j] *= decay;
      sk[j] = fmaf(ki, st[u].v[j], sk[j]);
      sq[j] = fmaf(qi, st[u].v[j], sq[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    sums[0][ty][tx * V + j] = sk[j];
    sums[1][ty][tx * V + j] = sq[j];
  }
  __syncthreads();
  // the columns' sums: 8 warps, a part of the rows each, then one warp
  if (tid < 2 * kSlice) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < TY; ++w) s += sums[tid / kSlice][w][tid % kSlice];
    out[tid / kSlice][tid % kSlice] = s;
  }
  __syncthreads();
  if (tid < ncol) {
    float dot = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) dot += kq_part[w];
    const float u = beta * (value - out[0][tid]);
    o[tid] = from_f32<T>(a.scale * fmaf(dot, u, out[1][tid]));
    out[0][tid] = u;
  }
  __syncthreads();
  if (!mine) return;
  float u[V];
#pragma unroll
  for (int j = 0; j < V; ++j) u[j] = out[0][tx * V + j];
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const int i = ty + w * TY;
    if (i >= a.dk) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) st[w].v[j] = fmaf(ks[i], u[j], st[w].v[j]);
    store_pack<float, V>(S + (size_t)i * a.dv, st[w]);
  }
}

template <typename T, int V>
void launch(const GdStepArgs& a, cudaStream_t s) {
  constexpr int TY = kThreads / (kSlice / V);
  const dim3 grid(a.B * a.H, (a.dv + kSlice - 1) / kSlice);
  if (a.dk <= 64) gd_step_kernel<T, V, 64 / TY><<<grid, kThreads, 0, s>>>(a);
  else if (a.dk <= 128) gd_step_kernel<T, V, 128 / TY><<<grid, kThreads, 0, s>>>(a);
  else gd_step_kernel<T, V, 256 / TY><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_gd_step(const GdStepArgs& a, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  const bool vec = a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  if (vec) {
    PRNN_BY_DTYPE(a.dtype, T, (launch<T, 4>(a, s)));
  } else {
    PRNN_BY_DTYPE(a.dtype, T, (launch<T, 1>(a, s)));
  }
  return cudaGetLastError();
}

}  // namespace prnn
