// linear_attention.cu -- linear attention with a decay per head over whole
// sequences: the `mix` operation of seq_internal.h in all its roles, for any
// sizes, strides and types.
//
// Unrolling S_t = l S_{t-1} + b_t c_t^T over a chunk of n tokens entered with
// state X gives
//   out_i = sum_{j<=i} l^(i-j) (a_i . b_j) c_j + l^(i+1) X^T a_i,
//   X'    = l^n X + sum_j l^(n-1-j) b_j c_j^T,
// so a chunk is four small matrix products and only the chunks are serial.
// Every exponent is >= 0: no power of the decay can overflow, whatever the
// decay, which factoring l^(i-j) into l^i l^-j would not give.
#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

constexpr int kChunk = 32, kCols = 32, kThreads = 256;

__device__ __forceinline__ int seq_len(const LaArgs& a, int b) {
  if (!a.lens) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

template <typename T>
__device__ __forceinline__ const T* seq_row(const LaSeq& s, long long t, int b, int h) {
  return static_cast<const T*>(s.p) + t * s.st + b * s.sb + (h / s.share) * s.sh;
}

// One block: one role, one (sequence, head) and kCols of the e columns.
template <typename T>
__global__ void __launch_bounds__(kThreads) la_mix_kernel(const __grid_constant__ LaArgs g) {
  const LaRole& r = g.role[blockIdx.z];
  const int col0 = blockIdx.y * kCols;
  if (col0 >= r.e) return;
  const int bh = blockIdx.x, b = bh / g.H, h = bh % g.H, d = r.d, tid = threadIdx.x;
  const int len = seq_len(g, b), ncol = min(kCols, r.e - col0);
  extern __shared__ float sm[];
  float* A = sm;                       // [kChunk][d + 1]
  float* Bm = A + kChunk * (d + 1);    // [kChunk][d + 1]
  float* Cm = Bm + kChunk * (d + 1);   // [kChunk][kCols]
  float* P = Cm + kChunk * kCols;      // [kChunk][kChunk + 1]
  float* X = P + kChunk * (kChunk + 1);  // [d][kCols]
  float* pw = X + d * kCols;           // [kChunk + 1]
  const float ld = g.log_decay[h];
  if (tid <= kChunk) pw[tid] = decay_pow(ld, tid);
  for (int i = tid; i < d * kCols; i += kThreads) {
    const int k = i / kCols, c = i % kCols;
    float v = 0.f;
    if (r.x0 && c < ncol)
      v = r.x0[(size_t)bh * d * r.e + (r.x_t ? (size_t)(col0 + c) * d + k
                                             : (size_t)k * r.e + col0 + c)];
    X[i] = v;
  }
  const int chunks = (len + kChunk - 1) / kChunk;
  for (int ci = 0; ci < chunks; ++ci) {
    const int t0 = (r.rev ? chunks - 1 - ci : ci) * kChunk, n = min(kChunk, len - t0);
    __syncthreads();
    for (int i = tid; i < kChunk * d; i += kThreads) {
      const int j = i / d, k = i % d;
      A[j * (d + 1) + k] = j < n ? to_f32(seq_row<T>(r.a, t0 + j, b, h)[k]) : 0.f;
      Bm[j * (d + 1) + k] = j < n ? to_f32(seq_row<T>(r.b, t0 + j, b, h)[k]) : 0.f;
    }
    for (int i = tid; i < kChunk * kCols; i += kThreads) {
      const int j = i / kCols, c = i % kCols;
      Cm[i] = j < n && c < ncol ? to_f32(seq_row<T>(r.c, t0 + j, b, h)[col0 + c]) : 0.f;
    }
    __syncthreads();
    for (int p = tid; p < kChunk * kChunk; p += kThreads) {
      const int i = p / kChunk, j = p % kChunk;
      float s = 0.f;
      if (r.rev ? j >= i : j <= i) {
        for (int k = 0; k < d; ++k) s = fmaf(A[i * (d + 1) + k], Bm[j * (d + 1) + k], s);
        s *= pw[r.rev ? j - i : i - j];
      }
      P[i * (kChunk + 1) + j] = s;
    }
    __syncthreads();
    for (int p = tid; p < n * kCols; p += kThreads) {
      const int i = p / kCols, c = p % kCols;
      float intra = 0.f, inter = 0.f;
      for (int j = 0; j < n; ++j) intra = fmaf(P[i * (kChunk + 1) + j], Cm[j * kCols + c], intra);
      for (int k = 0; k < d; ++k) inter = fmaf(A[i * (d + 1) + k], X[k * kCols + c], inter);
      const float v = r.s_intra * intra + r.s_inter * pw[(r.rev ? n - 1 - i : i) + r.lead] * inter;
      if (r.out && c < ncol) {
        const long long at = (long long)(t0 + i) * r.ot + b * r.ob + h * r.oh + col0 + c;
        if (r.out_f32)
          static_cast<float*>(r.out)[at] = v;
        else
          static_cast<T*>(r.out)[at] = from_f32<T>(v);
      }
    }
    __syncthreads();
    for (int p = tid; p < d * kCols; p += kThreads) {
      const int k = p / kCols, c = p % kCols;
      float s = 0.f;
      for (int j = 0; j < n; ++j)
        s = fmaf(Bm[j * (d + 1) + k] * pw[(r.rev ? j : n - 1 - j) + 1 - r.lead], Cm[j * kCols + c], s);
      X[p] = pw[n] * X[p] + r.s_add * s;
    }
  }
  __syncthreads();
  if (r.x_end)
    for (int i = tid; i < d * kCols; i += kThreads) {
      const int k = i / kCols, c = i % kCols;
      if (c < ncol)
        r.x_end[(size_t)bh * d * r.e + (r.x_t ? (size_t)(col0 + c) * d + k
                                              : (size_t)k * r.e + col0 + c)] = X[i];
    }
  if (r.out)
    for (long long p = tid; p < (long long)(g.T - len) * ncol; p += kThreads) {
      const long long at = (len + p / ncol) * r.ot + b * r.ob + h * r.oh + col0 + p % ncol;
      if (r.out_f32)
        static_cast<float*>(r.out)[at] = 0.f;
      else
        static_cast<T*>(r.out)[at] = from_f32<T>(0.f);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) la_reduce_kernel(LaReduceArgs a) {
  const int hq = a.H / a.group;
  const long long n = (long long)a.T * a.B * hq * a.d;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const int k = (int)(i % a.d), h = (int)(i / a.d % hq), b = (int)(i / a.d / hq % a.B);
    const long long t = i / a.d / hq / a.B;
    const float* p = a.part + ((t * a.B + b) * a.H + (long long)h * a.group) * a.d + k;
    float s = 0.f;
    for (int j = 0; j < a.group; ++j) s += p[(long long)j * a.d];
    static_cast<T*>(a.out)[t * a.ot + b * a.ob + h * a.oh + k] = from_f32<T>(s);
  }
}

size_t mix_smem(int d) {
  return sizeof(float) * (2 * kChunk * (d + 1) + kChunk * kCols + kChunk * (kChunk + 1) +
                          d * kCols + kChunk + 1);
}

}  // namespace

cudaError_t launch_la_simt(const LaArgs& a, cudaStream_t s) {
  int d = 0, e = 0;
  for (int i = 0; i < a.roles; ++i) {
    d = a.role[i].d > d ? a.role[i].d : d;
    e = a.role[i].e > e ? a.role[i].e : e;
  }
  if (a.roles == 0 || a.B == 0) return cudaSuccess;
  const size_t smem = mix_smem(d);
  const dim3 grid(a.B * a.H, (e + kCols - 1) / kCols, a.roles);
  cudaError_t err = cudaSuccess;
  PRNN_BY_DTYPE(a.dtype, T,
                err = cudaFuncSetAttribute(la_mix_kernel<T>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
                if (err == cudaSuccess) la_mix_kernel<T><<<grid, kThreads, smem, s>>>(a));
  return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_la_reduce(const LaReduceArgs& a, cudaStream_t s) {
  const long long n = (long long)a.T * a.B * (a.H / a.group) * a.d;
  if (n == 0) return cudaSuccess;
  const long long want = (n + 255) / 256;
  const int blocks = (int)(want < 152 * 16 ? want : 152 * 16);
  PRNN_BY_DTYPE(a.dtype, T, (la_reduce_kernel<T><<<blocks, 256, 0, s>>>(a)));
  return cudaGetLastError();
}

}  // namespace prnn
