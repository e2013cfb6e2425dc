// rms_api.cu -- the C ABI of root-mean-square norm: argument checks.  Contracts are in include/prnn.h.
#include <cmath>

#include "seq_checks.h"

using namespace prnn;

namespace {

struct Extent {
  const void* p;
  size_t n;
};
// Rows of a tensor: its bytes, or false where the pointer, the stride or the extent is no such tensor.
bool rows_ok(const void* p, long long rows, int cols, long long stride, size_t esz, Extent* e) {
  if (!p || !aligned(p, esz) || (rows > 1 && stride < cols)) return false;
  const long long n = row_extent(rows, cols, rows > 1 ? stride : cols);
  *e = {p, (size_t)n * esz};
  return n >= 0;
}
bool same_rows(const void* p, long long ps, const void* q, long long qs, long long rows) {
  return p == q && (rows == 1 || ps == qs);
}
bool meet(const Extent& a, const Extent& b) { return a.p && b.p && overlaps(a.p, a.n, b.p, b.n); }

prnn_status_t forward(RmsNormArgs a, bool quantised, void* stream) {
  if (!known(a.dtype) || a.rows < 0 || a.cols < 1 || !(a.eps >= 0.f) || !std::isfinite(a.eps))
    return PRNN_ERR_INVALID_ARG;
  if (quantised && a.group != 0 && a.group != 128) return PRNN_ERR_INVALID_ARG;
  if (a.rows == 0) return PRNN_OK;
  const size_t esz = elem_size(a.dtype);
  Extent x{}, res{}, y{}, h{};
  if (!rows_ok(a.x, a.rows, a.cols, a.x_stride, esz, &x) ||
      !rows_ok(a.y, a.rows, a.cols, a.y_stride, quantised ? 1 : esz, &y) ||
      (a.residual && (!rows_ok(a.residual, a.rows, a.cols, a.residual_stride, esz, &res) ||
                      !rows_ok(a.h, a.rows, a.cols, a.h_stride, esz, &h))) ||
      !aligned(a.weight, 4) || !aligned(a.rstd, 4) || !aligned(a.scale, 4) || (quantised && !a.scale))
    return PRNN_ERR_INVALID_ARG;
  if (!a.residual) a.h = nullptr;  // the stream is x itself: nothing is written
  if (a.rows > LLONG_MAX / 64) return PRNN_ERR_INVALID_ARG;
  const long long groups = quantised && a.group ? (a.cols + (long long)a.group - 1) / a.group : 1;
  size_t scales;
  if (__builtin_mul_overflow((size_t)a.rows, (size_t)groups * 4, &scales)) return PRNN_ERR_INVALID_ARG;
  // a row may be written over the one it was read from, where both hold the same type
  const Extent w{a.weight, 4ull * a.cols}, rstd{a.rstd, 4ull * a.rows}, scale{a.scale, scales};
  if ((meet(h, x) && !same_rows(a.h, a.h_stride, a.x, a.x_stride, a.rows)) ||
      (meet(h, res) && !same_rows(a.h, a.h_stride, a.residual, a.residual_stride, a.rows)) ||
      (meet(y, x) && (quantised || !same_rows(a.y, a.y_stride, a.x, a.x_stride, a.rows))) ||
      (meet(y, res) && (quantised || !same_rows(a.y, a.y_stride, a.residual, a.residual_stride, a.rows))))
    return PRNN_ERR_INVALID_ARG;
  const Extent outs[] = {y, h, rstd, scale};
  for (int i = 0; i < 4; ++i) {
    if (meet(outs[i], w) || (i >= 2 && (meet(outs[i], x) || meet(outs[i], res)))) return PRNN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return PRNN_ERR_INVALID_ARG;
  }
  return cuda_status(launch_rms_norm(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

prnn_status_t prnn_rms_norm_forward(prnn_dtype_t dtype, long long rows, int cols, const void* x, long long x_stride,
                                    const void* residual, long long residual_stride, const float* weight, float eps,
                                    void* y, long long y_stride, void* h, long long h_stride, float* rstd,
                                    void* stream) {
  return forward({dtype, rows, cols, x, x_stride, residual, residual_stride, weight, eps, y, y_stride, h, h_stride,
                  rstd, 0, nullptr}, false, stream);
}

prnn_status_t prnn_rms_norm_quantized(prnn_dtype_t dtype, long long rows, int cols, const void* x,
                                         long long x_stride, const void* residual, long long residual_stride,
                                         const float* weight, float eps, int group, void* q, long long q_stride,
                                         float* scale, void* h, long long h_stride, float* rstd, void* stream) {
  return forward({dtype, rows, cols, x, x_stride, residual, residual_stride, weight, eps, q, q_stride, h, h_stride,
                  rstd, group, scale}, true, stream);
}

prnn_status_t prnn_rms_norm_workspace(long long rows, int cols, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 1) return PRNN_ERR_INVALID_ARG;
  *bytes = (sizeof(float) * (size_t)rms_norm_splits(rows, cols) * cols + 15) / 16 * 16;
  return PRNN_OK;
}

prnn_status_t prnn_rms_norm_backward(prnn_dtype_t dtype, long long rows, int cols, const void* dy,
                                     long long dy_stride, const void* h, long long h_stride, const float* weight,
                                     const float* rstd, const void* dh, long long dh_stride, void* dx,
                                     long long dx_stride, float* dweight, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!known(dtype) || rows < 0 || cols < 1 || !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(dweight, 4))
    return PRNN_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dweight) PRNN_TRY(cudaMemsetAsync(dweight, 0, 4ull * cols, s));
    return PRNN_OK;
  }
  const size_t esz = elem_size(dtype);
  Extent ey{}, eh{}, ed{}, ex{};
  if (!rstd || rows > LLONG_MAX / 64 || !rows_ok(dy, rows, cols, dy_stride, esz, &ey) ||
      !rows_ok(h, rows, cols, h_stride, esz, &eh) || (dh && !rows_ok(dh, rows, cols, dh_stride, esz, &ed)) ||
      (dx && !rows_ok(dx, rows, cols, dx_stride, esz, &ex)))
    return PRNN_ERR_INVALID_ARG;
  size_t need = 0;
  prnn_rms_norm_workspace(rows, cols, &need);
  if (dweight && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return PRNN_ERR_INVALID_ARG;
  if ((meet(ex, ey) && !same_rows(dx, dx_stride, dy, dy_stride, rows)) ||
      (meet(ex, ed) && !same_rows(dx, dx_stride, dh, dh_stride, rows)))
    return PRNN_ERR_INVALID_ARG;
  const Extent ins[] = {eh, {weight, 4ull * cols}, {rstd, 4ull * rows}, ey, ed};
  const Extent outs[] = {ex, {dweight, 4ull * cols}, {dweight ? workspace : nullptr, need}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < (i == 0 ? 3 : 5); ++j)
      if (meet(outs[i], ins[j])) return PRNN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return PRNN_ERR_INVALID_ARG;
  }
  if (!dx && !dweight) return PRNN_OK;
  return cuda_status(launch_rms_norm_grad({dtype, rows, cols, dy, h, dh, dy_stride, h_stride, dh_stride, weight, rstd,
                                           dx, dx_stride, dweight, static_cast<float*>(workspace)}, s));
}

}  // extern "C"
