// seq_internal.h -- what the sequence operators (layer norm, dropout, linear
// attention) share between their C ABI checks (seq_api.cu) and their kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "prnn.h"

namespace prnn {

// The current device's status word of the sequence operators (device int, 0 = no wait has run out);
// nullptr when it cannot be had.  Looked up at every call, so it survives a device reset.
int* seq_status_word();
// SMs of the current device (1 when unknown).
int seq_sm_count();

// ---- layer norm (layer_norm.cu) -------------------------------------------
struct LayerNormArgs {
  prnn_dtype_t dtype;
  long long rows;
  int cols;
  const void* x;
  long long x_stride;
  const float *gamma, *beta;  // may be null
  float eps;
  void* y;
  long long y_stride;
  float *mean, *rstd;         // may be null
};
cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s);

struct LayerNormGradArgs {
  prnn_dtype_t dtype;
  long long rows;
  int cols;
  const void *dy, *x;
  long long dy_stride, x_stride;
  const float *gamma, *mean, *rstd;
  void* dx;                   // may be null
  long long dx_stride;
  float *dgamma, *dbeta;      // may be null
  float* partial;             // [2][layer_norm_splits][cols]
};
// Row blocks whose partial sums of dgamma and dbeta are kept apart.
int layer_norm_splits(long long rows, int cols);
cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& a, cudaStream_t s);

// ---- root-mean-square norm (rms_norm.cu) ------------------------------------
struct RmsNormArgs {
  prnn_dtype_t dtype;
  long long rows;
  int cols;
  const void* x;
  long long x_stride;
  const void* residual;       // may be null, and then h is
  long long residual_stride;
  const float* weight;        // may be null
  float eps;
  void* y;                    // dtype, or bytes of e4m3 where scale is set
  long long y_stride;
  void* h;
  long long h_stride;
  float* rstd;                // may be null
  int group;                  // columns of one scale: 128, or 0 for the row
  float* scale;
};
cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t s);

struct RmsNormGradArgs {
  prnn_dtype_t dtype;
  long long rows;
  int cols;
  const void *dy, *h, *dh;    // dh may be null
  long long dy_stride, h_stride, dh_stride;
  const float *weight, *rstd;
  void* dx;                   // may be null
  long long dx_stride;
  float* dweight;             // may be null
  float* partial;             // [rms_norm_splits][cols]
};
int rms_norm_splits(long long rows, int cols);
cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, cudaStream_t s);

// ---- dropout (dropout.cu) ---------------------------------------------------
struct DropoutArgs {
  prnn_dtype_t dtype;
  long long n;
  const void *x, *residual;   // residual may be null
  void* y;
  uint32_t limit;             // a word below it drops its value
  float scale;                // 1 / (1 - p)
  uint64_t seed, offset;
};
cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t s);

// ---- linear attention -------------------------------------------------------
// Forward and backward are one operation, `mix`, in different roles: with a, b, c
// sequences of d, d and e values per token and X a d x e state,
//   out_i = s_intra sum_j l^|i-j| (a_i . b_j) c_j + s_inter l^(.) X^T a_i,
//   X    <- l^n X + s_add sum_j l^(.) b_j c_j^T,
// j running over the tokens not after i (rev = 0) or not before it (rev = 1).
//   forward: a, b, c = q, k, v;  dq: do, v, k;  dk: v, do, q (rev);  dv: k, q, do (rev).
// lead: the power of l the entering state has at the first token, 1 in the
// forward direction (S before the token, decayed once by it) and 0 in reverse
// (the carried state has the decay already applied).
struct LaSeq {
  const void* p;
  long long st, sb, sh;
  int share;                  // heads that share one head of this tensor
};
struct LaRole {
  LaSeq a, b, c;
  void* out;                  // may be null
  long long ot, ob, oh;
  int out_f32;                // 1: out is fp32 whatever the dtype (summed over heads later)
  int d, e;
  const float* x0;            // state entering, may be null (zeros)
  float* x_end;               // state leaving, may be null
  int x_t;                    // 1: x0 and x_end hold [e][d] per head instead of [d][e]
  int rev, lead;
  float s_intra, s_inter, s_add;
};
struct LaArgs {
  LaRole role[3];
  int roles;
  prnn_dtype_t dtype;
  int T, B, H;
  const float* log_decay;
  const int32_t* lens;        // may be null
};
// On CUDA cores, for any sizes, strides and types.
size_t la_simt_workspace(const LaArgs& a);
cudaError_t launch_la_simt(const LaArgs& a, void* scratch, size_t bytes, cudaStream_t s);
// On the tensor cores, for fp16 and bf16 with d, e <= 128: whether it serves a call; the bytes of scratch for
// its segments' states and for a copy of an input that it cannot read in place (0: it can); the call.
bool la_tc_serves(const LaArgs& a);
size_t la_tc_workspace(const LaArgs& a);
size_t la_tc_copy_bytes(const LaSeq& x, const LaArgs& a, int d);
cudaError_t launch_la_tc(const LaArgs& a, void* scratch, size_t bytes, cudaStream_t s);

// out[t][b][hq][:] = sum of the `group` heads of part [T][B][H][d] (fp32) that share hq.
struct LaReduceArgs {
  prnn_dtype_t dtype;
  const float* part;
  void* out;
  long long ot, ob, oh;
  int T, B, H, group, d;
};
cudaError_t launch_la_reduce(const LaReduceArgs& a, cudaStream_t s);

struct LaStepArgs {
  prnn_dtype_t dtype;
  int B, H, dk, dv;
  LaSeq q, k, v;
  void* o;
  long long ob, oh;
  const float* log_decay;
  float* state;
  int n_slots;
  const int32_t* slots;       // may be null
  float scale;
};
cudaError_t launch_la_step(const LaStepArgs& a, cudaStream_t s);

}  // namespace prnn
