// gated_delta_api.cu -- the C ABI of the gated delta rule: argument checks and the division of workspaces.
// Contracts are in include/prnn.h.
#include <cmath>

#include "gated_delta.h"
#include "seq_checks.h"

using namespace prnn;

namespace {

using Call = prnn_gated_delta_t;

bool shape_ok(const Call* a, prnn_status_t* why) {
  *why = PRNN_ERR_INVALID_ARG;
  if (!a || !known(a->dtype) || a->T < 0 || a->B < 0 || a->heads < 1 || a->qk_heads < 1 ||
      a->heads % a->qk_heads != 0 || a->dk < 1 || a->dv < 1 || !std::isfinite(a->scale))
    return false;
  if (a->dk > 256 || a->dv > 256 || a->T > (1 << 29) || (long long)a->B * a->heads > (1 << 24)) {
    *why = PRNN_ERR_UNSUPPORTED;
    return false;
  }
  *why = PRNN_OK;
  return true;
}

// A tensor or plain array of a call.
struct Area {
  const void* p;
  Dims d;
  size_t esz;
  bool out, in_place;
};
struct Areas {
  Area at[24];
  int n = 0;
  bool ok = true;
  void tensor(const prnn_seq_t& x, int T, int B, int H, int w, size_t esz, bool out) {
    if (out && !x.data) return;
    const Area a{x.data, dims_of(x, T, B, H, w), esz, out, false};
    ok = ok && seq_ok(x, a.d, esz, out);
    at[n++] = a;
  }
  // in_place: may lie exactly upon the other array of that kind
  void array(const void* p, size_t bytes, bool out, bool in_place = false) {
    if (!p || !bytes) return;
    ok = ok && aligned(p, 4);
    at[n++] = {p, Dims{{1, 1, (long long)(bytes / 4)}, {0, 0, 1}, 1}, 4, out, in_place};
  }
  bool meet(const Area& a, const Area& b) const {
    if (a.esz == b.esz) return !apart(a.p, a.d, b.p, b.d, a.esz);
    return overlaps(a.p, (size_t)span(a.d, 0) * a.esz, b.p, (size_t)span(b.d, 0) * b.esz);
  }
  // Every part is a tensor, and no output meets anything else.
  bool good() const {
    if (!ok) return false;
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j)
        if (i != j && at[i].out && (!at[j].out || i < j) &&
            !(at[i].in_place && at[j].in_place && at[i].p == at[j].p) && meet(at[i], at[j]))
          return false;
    return true;
  }
};

size_t state_bytes(const Call* a) { return sizeof(float) * (size_t)a->B * a->heads * a->dk * a->dv; }

void inputs(Areas& all, const Call* a, int T) {
  all.tensor(a->q, T, a->B, a->qk_heads, a->dk, elem_size(a->dtype), false);
  all.tensor(a->k, T, a->B, a->qk_heads, a->dk, elem_size(a->dtype), false);
  all.tensor(a->v, T, a->B, a->heads, a->dv, elem_size(a->dtype), false);
  all.tensor(a->log_decay, T, a->B, a->heads, 1, 4, false);
  all.tensor(a->beta, T, a->B, a->heads, 1, 4, false);
}

// The walks' scratch, in floats.
struct Parts {
  size_t e, dq, marks, leaves, total;
};
size_t round16(size_t bytes) { return (bytes + 15) / 16 * 16; }
Parts walk_parts(const Call* a) {
  const size_t tokens = (size_t)a->T * a->B * a->heads, blocks = ((size_t)a->T + kGdBlock - 1) / kGdBlock;
  Parts p;
  p.e = round16(4 * tokens * a->dv);
  p.dq = round16(4 * tokens * a->dk);
  p.marks = round16(4 * blocks * a->B * a->heads * a->dk * a->dv);
  p.leaves = round16(4 * blocks * a->B * a->heads * a->dk);
  p.total = 2 * p.e + 2 * p.dq + p.marks + p.leaves;
  return p;
}

bool on_tensor_cores(const Call* a, bool backward) {
  return gd_tc_serves(a->T, a->B, a->heads, a->dk, a->dv, backward);
}

GdArgs args_of(const Call* a) {
  GdArgs g{};
  g.dtype = a->dtype;
  g.T = a->T;
  g.B = a->B;
  g.H = a->heads;
  g.dk = a->dk;
  g.dv = a->dv;
  g.scale = a->scale;
  g.g = static_cast<const float*>(a->log_decay.data);
  g.gt = a->log_decay.stride_t;
  g.gb = a->log_decay.stride_b;
  g.gh = a->log_decay.stride_h;
  g.beta = static_cast<const float*>(a->beta.data);
  g.bt = a->beta.stride_t;
  g.bb = a->beta.stride_b;
  g.bh = a->beta.stride_h;
  g.lens = a->lens;
  const int share = a->heads / a->qk_heads;
  g.q = in(a->q, share);
  g.k = in(a->k, share);
  g.v = in(a->v, 1);
  g.state = a->state;
  g.o = a->o.data;
  g.ot = a->o.stride_t;
  g.ob = a->o.stride_b;
  g.oh = a->o.stride_h;
  g.state_out = a->state_out;
  g.d_o = in(a->d_o, 1);
  g.d_state_out = a->d_state_out;
  g.d_state = a->d_state;
  g.dq_out = a->d_q.data;
  g.dqt = a->d_q.stride_t;
  g.dqb = a->d_q.stride_b;
  g.dqh = a->d_q.stride_h;
  g.dk_out = a->d_k.data;
  g.dkt = a->d_k.stride_t;
  g.dkb = a->d_k.stride_b;
  g.dkh = a->d_k.stride_h;
  g.dv_out = a->d_v.data;
  g.dvt = a->d_v.stride_t;
  g.dvb = a->d_v.stride_b;
  g.dvh = a->d_v.stride_h;
  g.dg = static_cast<float*>(a->d_log_decay.data);
  g.dgt = a->d_log_decay.stride_t;
  g.dgb = a->d_log_decay.stride_b;
  g.dgh = a->d_log_decay.stride_h;
  g.dbeta = static_cast<float*>(a->d_beta.data);
  g.dbt = a->d_beta.stride_t;
  g.dbb = a->d_beta.stride_b;
  g.dbh = a->d_beta.stride_h;
  return g;
}

}  // namespace

extern "C" {

prnn_status_t prnn_gated_delta_workspace(const prnn_gated_delta_t* a, int backward, size_t* bytes) {
  prnn_status_t why;
  if (!bytes) return PRNN_ERR_INVALID_ARG;
  if (!shape_ok(a, &why)) return why;
  *bytes = 0;
  if (a->T == 0 || a->B == 0) return PRNN_OK;
  if (on_tensor_cores(a, backward != 0)) *bytes = gd_tc_workspace(args_of(a), backward != 0);
  else if (backward) *bytes = walk_parts(a).total;
  return PRNN_OK;
}

prnn_status_t prnn_gated_delta_forward(const prnn_gated_delta_t* a, void* stream) {
  prnn_status_t why;
  if (!shape_ok(a, &why)) return why;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->B == 0) return PRNN_OK;
  const size_t sb = state_bytes(a);
  Areas all;
  all.array(a->state, sb, false, true);
  all.array(a->state_out, sb, true, true);
  if (a->T == 0) {
    if (!all.good()) return PRNN_ERR_INVALID_ARG;
    if (!a->state_out || a->state_out == a->state) return PRNN_OK;
    if (a->state) return cuda_status(cudaMemcpyAsync(a->state_out, a->state, sb, cudaMemcpyDeviceToDevice, s));
    return cuda_status(cudaMemsetAsync(a->state_out, 0, sb, s));
  }
  size_t need = 0;
  prnn_gated_delta_workspace(a, 0, &need);
  if (need && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need)) return PRNN_ERR_INVALID_ARG;
  inputs(all, a, a->T);
  if (!a->o.data) return PRNN_ERR_INVALID_ARG;
  all.tensor(a->o, a->T, a->B, a->heads, a->dv, elem_size(a->dtype), true);
  all.array(a->lens, 4ull * a->B, false);
  if (need) all.array(a->workspace, need, true);
  if (!all.good()) return PRNN_ERR_INVALID_ARG;
  GdArgs g = args_of(a);
  return cuda_status(on_tensor_cores(a, false) ? launch_gd_tc(g, a->workspace, false, s) : launch_gd_walk_forward(g, s));
}

prnn_status_t prnn_gated_delta_backward(const prnn_gated_delta_t* a, void* stream) {
  prnn_status_t why;
  if (!shape_ok(a, &why)) return why;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->B == 0) return PRNN_OK;
  const size_t sb = state_bytes(a);
  Areas all;
  all.array(a->state, sb, false);
  all.array(a->d_state_out, sb, false);
  all.array(a->d_state, sb, true);
  if (a->T == 0) {
    if (!all.good()) return PRNN_ERR_INVALID_ARG;
    if (!a->d_state) return PRNN_OK;
    if (a->d_state_out) return cuda_status(cudaMemcpyAsync(a->d_state, a->d_state_out, sb, cudaMemcpyDeviceToDevice, s));
    return cuda_status(cudaMemsetAsync(a->d_state, 0, sb, s));
  }
  size_t need = 0;
  prnn_gated_delta_workspace(a, 1, &need);
  if (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need) return PRNN_ERR_INVALID_ARG;
  const size_t esz = elem_size(a->dtype);
  const int T = a->T, B = a->B, H = a->heads, Hq = a->qk_heads;
  inputs(all, a, T);
  all.tensor(a->d_o, T, B, H, a->dv, esz, false);
  all.tensor(a->d_q, T, B, Hq, a->dk, esz, true);
  all.tensor(a->d_k, T, B, Hq, a->dk, esz, true);
  all.tensor(a->d_v, T, B, H, a->dv, esz, true);
  all.tensor(a->d_log_decay, T, B, H, 1, 4, true);
  all.tensor(a->d_beta, T, B, H, 1, 4, true);
  all.array(a->lens, 4ull * B, false);
  all.array(a->workspace, need, true);
  if (!all.good()) return PRNN_ERR_INVALID_ARG;
  GdArgs g = args_of(a);
  // the forward call's outputs, which a descriptor of both passes still names: the kernels of the forward pass, which run
  // again here, write them where they are given
  g.o = nullptr;
  g.state_out = nullptr;
  if (on_tensor_cores(a, true)) return cuda_status(launch_gd_tc(g, a->workspace, true, s));
  const Parts p = walk_parts(a);
  char* w = static_cast<char*>(a->workspace);
  auto take = [&](size_t n) {
    float* at = reinterpret_cast<float*>(w);
    w += n;
    return at;
  };
  g.e = take(p.e);
  g.du = take(p.e);
  g.dq_part = take(p.dq);
  g.dk_part = take(p.dq);
  g.marks = take(p.marks);
  g.leaves = take(p.leaves);
  PRNN_TRY(launch_gd_walk_backward(g, s));
  const prnn_seq_t* out[] = {&a->d_q, &a->d_k};
  const float* part[] = {g.dq_part, g.dk_part};
  for (int i = 0; i < 2; ++i)
    if (out[i]->data)
      PRNN_TRY(launch_la_reduce({a->dtype, part[i], out[i]->data, out[i]->stride_t, out[i]->stride_b,
                                 out[i]->stride_h, T, B, H, H / Hq, a->dk}, s));
  return PRNN_OK;
}

prnn_status_t prnn_gated_delta_step(const prnn_gated_delta_t* a, float* state_pool, int n_slots,
                                    const int32_t* slots, void* stream) {
  prnn_status_t why;
  if (!shape_ok(a, &why)) return why;
  if (n_slots < 0) return PRNN_ERR_INVALID_ARG;
  if (a->B == 0) return PRNN_OK;
  if (!state_pool || !aligned(slots, 4) || (!slots && n_slots < a->B) || !a->o.data) return PRNN_ERR_INVALID_ARG;
  Call one = *a;
  for (prnn_seq_t* x : {&one.q, &one.k, &one.v, &one.o, &one.log_decay, &one.beta}) x->stride_t = 0;
  Areas all;
  inputs(all, &one, 1);
  all.tensor(one.o, 1, a->B, a->heads, a->dv, elem_size(a->dtype), true);
  all.array(state_pool, sizeof(float) * (size_t)n_slots * a->heads * a->dk * a->dv, true);
  all.array(slots, 4ull * a->B, false);
  if (!all.good()) return PRNN_ERR_INVALID_ARG;
  const GdArgs g = args_of(&one);
  GdStepArgs r{a->dtype, a->B, a->heads, a->dk, a->dv, a->scale, g.g, g.beta, g.gb, g.gh, g.bb, g.bh, g.q, g.k, g.v,
               one.o.data, one.o.stride_b, one.o.stride_h, state_pool, n_slots, slots};
  return cuda_status(launch_gd_step(r, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
