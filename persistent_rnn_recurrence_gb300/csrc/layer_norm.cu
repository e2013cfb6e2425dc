// layer_norm.cu -- layer norm over the last axis and its gradient.
//
// Both are bound by memory: 8 to 14 flops per element against 4 to 12 bytes.
#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

// One block per row.  The mean is taken first and the squared distances from
// it next: E[x^2] - mean^2 would lose the variance of rows whose mean is large.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_kernel(LayerNormArgs a) {
  __shared__ float part[2][8];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    T* y = static_cast<T*>(a.y) + r * a.y_stride;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) s += to_f32(x[c]);
    const float mean = block_sum(s, part[0]) / a.cols;
    float q = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float d = to_f32(x[c]) - mean;
      q += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(q, part[1]) / a.cols + a.eps);
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = a.gamma ? a.gamma[c] : 1.f, b = a.beta ? a.beta[c] : 0.f;
      y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * g + b);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(256) layer_norm_dx_kernel(LayerNormGradArgs a) {
  __shared__ float part[2][8];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(dy[c]) * (a.gamma ? a.gamma[c] : 1.f);
      s += g;
      q += g * ((to_f32(x[c]) - mean) * rstd);
    }
    s = block_sum(s, part[0]) / a.cols;
    q = block_sum(q, part[1]) / a.cols;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(dy[c]) * (a.gamma ? a.gamma[c] : 1.f);
      dx[c] = from_f32<T>(rstd * (g - s - (to_f32(x[c]) - mean) * rstd * q));
    }
    __syncthreads();
  }
}

// Partial sums of dgamma and dbeta: block (x, y) sums 32 columns over the y-th share of the rows.
template <typename T>
__global__ void layer_norm_dw_kernel(LayerNormGradArgs a, int splits) {
  __shared__ float pg[32][33], pb[32][33];
  const int tx = threadIdx.x, ty = threadIdx.y, c = blockIdx.x * 32 + tx;
  const long long share = (a.rows + splits - 1) / splits;
  const long long lo = blockIdx.y * share, hi = lo + share < a.rows ? lo + share : a.rows;
  float g = 0.f, b = 0.f;
  if (c < a.cols)
    for (long long r = lo + ty; r < hi; r += 32) {
      const float d = to_f32(static_cast<const T*>(a.dy)[r * a.dy_stride + c]);
      g += d * (to_f32(static_cast<const T*>(a.x)[r * a.x_stride + c]) - a.mean[r]) * a.rstd[r];
      b += d;
    }
  pg[ty][tx] = g;
  pb[ty][tx] = b;
  __syncthreads();
  if (ty == 0 && c < a.cols) {
    g = b = 0.f;
    for (int i = 0; i < 32; ++i) {
      g += pg[i][tx];
      b += pb[i][tx];
    }
    a.partial[(size_t)blockIdx.y * a.cols + c] = g;
    a.partial[(size_t)(splits + blockIdx.y) * a.cols + c] = b;
  }
}

__global__ void layer_norm_dw_join_kernel(const float* partial, int splits, int cols,
                                          float* dgamma, float* dbeta) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float g = 0.f, b = 0.f;
  for (int i = 0; i < splits; ++i) {
    g += partial[(size_t)i * cols + c];
    b += partial[(size_t)(splits + i) * cols + c];
  }
  if (dgamma) dgamma[c] = g;
  if (dbeta) dbeta[c] = b;
}

}  // namespace

int layer_norm_splits(long long rows, int) {
  const long long s = (rows + 63) / 64;
  return (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const int blocks = (int)(a.rows < 65536 ? a.rows : 65536);
  PRNN_BY_DTYPE(a.dtype, T, (layer_norm_kernel<T><<<blocks, 256, 0, s>>>(a)));
  return cudaGetLastError();
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& a, cudaStream_t s) {
  if (a.dx && a.rows > 0) {
    const int blocks = (int)(a.rows < 65536 ? a.rows : 65536);
    PRNN_BY_DTYPE(a.dtype, T, (layer_norm_dx_kernel<T><<<blocks, 256, 0, s>>>(a)));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!a.dgamma && !a.dbeta) return cudaSuccess;
  const int splits = layer_norm_splits(a.rows, a.cols);
  const dim3 grid((a.cols + 31) / 32, splits);
  PRNN_BY_DTYPE(a.dtype, T, (layer_norm_dw_kernel<T><<<grid, dim3(32, 32), 0, s>>>(a, splits)));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  layer_norm_dw_join_kernel<<<(a.cols + 255) / 256, 256, 0, s>>>(a.partial, splits, a.cols,
                                                                 a.dgamma, a.dbeta);
  return cudaGetLastError();
}

}  // namespace prnn
