// gated_delta.h -- what the gated delta rule's C ABI checks (gated_delta_api.cu) and kernels share.
#pragma once

#include "seq_internal.h"

namespace prnn {

constexpr int kGdBlock = 128;  // tokens whose decays' gradients are summed together

struct GdArgs {
  prnn_dtype_t dtype;
  int T, B, H, dk, dv;
  float scale;
  const float *g, *beta;        // log-decays and betas, with their strides
  long long gt, gb, gh, bt, bb, bh;
  const int32_t* lens;          // may be null
  LaSeq q, k, v, d_o;
  const float* state;           // may be null
  void* o;                      // may be null
  long long ot, ob, oh;
  float* state_out;             // may be null
  const float* d_state_out;     // may be null
  void *dq_out, *dk_out, *dv_out;  // may be null
  long long dqt, dqb, dqh, dkt, dkb, dkh, dvt, dvb, dvh;
  float *dg, *dbeta;            // may be null
  long long dgt, dgb, dgh, dbt, dbb, dbh;
  float* d_state;               // may be null
  // scratch, fp32: [T][B][H][dv] e (null: not kept) and du, [T][B][H][dk] gradients before shared heads are summed,
  // the states at the ends of blocks [blocks][B*H][dk][dv] and their products with the gradients [blocks][B*H][dk]
  float *e, *du, *dq_part, *dk_part, *marks, *leaves;
  // tensor cores: rows rounded up to 8 values, and fp32 parts [T][B][H][dkp or dvp] of results that the kernels do not
  // write in place (dq_part and dk_part as well)
  int dkp, dvp;
  float *o_part, *dv_part;
};

cudaError_t launch_gd_walk_forward(const GdArgs& a, cudaStream_t s);
cudaError_t launch_gd_walk_backward(const GdArgs& a, cudaStream_t s);

// On the tensor cores, in chunks, for dk and dv up to 128: whether it serves a call, its scratch, the call.
bool gd_tc_serves(int T, int B, int H, int dk, int dv, bool backward);
size_t gd_tc_workspace(const GdArgs& a, bool backward);
cudaError_t launch_gd_tc(GdArgs a, void* scratch, bool backward, cudaStream_t s);

struct GdStepArgs {
  prnn_dtype_t dtype;
  int B, H, dk, dv;
  float scale;
  const float *g, *beta;
  long long gb, gh, bb, bh;
  LaSeq q, k, v;
  void* o;
  long long ob, oh;
  float* state;
  int n_slots;
  const int32_t* slots;         // may be null
};
cudaError_t launch_gd_step(const GdStepArgs& a, cudaStream_t s);

}  // namespace prnn
