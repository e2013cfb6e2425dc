// seq_api.cu -- the C ABI of the sequence operators: argument checks, the
// division of workspaces, and the roles of linear attention's forward and
// backward passes.  Contracts are in include/prnn.h.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "prnn.h"
#include "seq_checks.h"
#include "seq_internal.h"

using namespace prnn;

namespace prnn {

__device__ int g_seq_status;

int* seq_status_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_seq_status) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int seq_sm_count() {
  // a device's count never changes; kept because a short call would spend as long asking as launching
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace prnn

namespace {

bool shape_ok(const prnn_linear_attention_t* a, prnn_status_t* why) {
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

// What a call writes beside its sequence outputs must not overlap the small arrays it reads (the decays, and the
// lengths or slots): blocks read them while others write.
bool tables_clear(const void* p, size_t bytes, const prnn_linear_attention_t* a, const int32_t* per_sequence) {
  if (!p || !bytes) return true;
  return !overlaps(p, bytes, a->log_decay, sizeof(float) * (size_t)a->heads) &&
         (!per_sequence || !overlaps(p, bytes, per_sequence, sizeof(int32_t) * (size_t)a->B));
}

// Bytes of the fp32 partial gradients of heads that share a query and key head (one of dq and dk).
size_t group_bytes(const prnn_linear_attention_t* a) {
  if (a->heads == a->qk_heads) return 0;
  return (sizeof(float) * (size_t)a->T * a->B * a->heads * a->dk + 15) / 16 * 16;
}
// Bytes of the kernels' scratch for these sizes: any subset of the backward pass's roles fits.
size_t mix_bytes(const prnn_linear_attention_t* a, bool backward) {
  if (a->T == 0 || a->B == 0) return 0;
  LaArgs g{};
  g.dtype = a->dtype;
  g.T = a->T;
  g.B = a->B;
  g.H = a->heads;
  for (LaRole& r : g.role) {
    r.d = backward ? std::max(a->dk, a->dv) : a->dk;
    r.e = backward ? std::max(a->dk, a->dv) : a->dv;
  }
  g.roles = backward ? 3 : 1;
  const bool tc = la_tc_serves(g);
  size_t most = 0;
  for (g.roles = 1; g.roles <= (backward ? 3 : 1); ++g.roles)
    most = std::max(most, tc ? la_tc_workspace(g) : la_simt_workspace(g));
  if (!tc) return most;
  const int share = a->heads / a->qk_heads;
  most += la_tc_copy_bytes(in(a->q, share), g, a->dk) + la_tc_copy_bytes(in(a->k, share), g, a->dk) +
          la_tc_copy_bytes(in(a->v, 1), g, a->dv);
  if (backward) most += la_tc_copy_bytes(in(a->d_o, 1), g, a->dv);
  return most;
}
cudaError_t launch_mix(const LaArgs& g, void* scratch, size_t bytes, cudaStream_t s) {
  if (la_tc_serves(g)) return launch_la_tc(g, scratch, bytes, s);
  return launch_la_simt(g, scratch, bytes, s);
}

}  // namespace

extern "C" {

prnn_status_t prnn_sequence_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int v = 0;
  const int* p = seq_status_word();
  if (!p) return PRNN_ERR_CUDA;
  PRNN_TRY(cudaMemcpyAsync(&v, p, sizeof(int), cudaMemcpyDeviceToHost, s));
  PRNN_TRY(cudaStreamSynchronize(s));
  return v ? PRNN_ERR_TIMEOUT : PRNN_OK;
}

prnn_status_t prnn_layer_norm_forward(prnn_dtype_t dtype, long long rows, int cols, const void* x,
                                      long long x_stride, const float* gamma, const float* beta,
                                      float eps, void* y, long long y_stride, float* mean,
                                      float* rstd, void* stream) {
  if (!known(dtype) || rows < 0 || cols < 1 || !(eps >= 0.f) || !std::isfinite(eps))
    return PRNN_ERR_INVALID_ARG;
  if (rows == 0) return PRNN_OK;
  const size_t esz = elem_size(dtype);
  if (!x || !y || !aligned(x, esz) || !aligned(y, esz) || !aligned(gamma, 4) || !aligned(beta, 4) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return PRNN_ERR_INVALID_ARG;
  if (rows > 1 && (x_stride < cols || y_stride < cols)) return PRNN_ERR_INVALID_ARG;
  const long long nx = row_extent(rows, cols, rows > 1 ? x_stride : cols);
  const long long ny = row_extent(rows, cols, rows > 1 ? y_stride : cols);
  if (nx < 0 || ny < 0) return PRNN_ERR_INVALID_ARG;
  const bool in_place = x == y && (rows == 1 || x_stride == y_stride);
  if (!in_place && overlaps(x, nx * esz, y, ny * esz)) return PRNN_ERR_INVALID_ARG;
  struct { const void* p; size_t n; } par[2] = {{gamma, 4ull * cols}, {beta, 4ull * cols}},
      st[2] = {{mean, 4ull * rows}, {rstd, 4ull * rows}};
  for (auto& q : par)
    if (q.p && overlaps(q.p, q.n, y, ny * esz)) return PRNN_ERR_INVALID_ARG;
  for (auto& o : st) {
    if (!o.p) continue;
    if (overlaps(o.p, o.n, y, ny * esz) || overlaps(o.p, o.n, x, nx * esz))
      return PRNN_ERR_INVALID_ARG;
    for (auto& q : par)
      if (q.p && overlaps(q.p, q.n, o.p, o.n)) return PRNN_ERR_INVALID_ARG;
  }
  if (mean && rstd && overlaps(mean, 4 * rows, rstd, 4 * rows)) return PRNN_ERR_INVALID_ARG;
  LayerNormArgs a{dtype, rows, cols, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd};
  return cuda_status(launch_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

prnn_status_t prnn_layer_norm_workspace(long long rows, int cols, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 1) return PRNN_ERR_INVALID_ARG;
  *bytes = 2 * sizeof(float) * (size_t)layer_norm_splits(rows, cols) * cols;
  return PRNN_OK;
}

prnn_status_t prnn_layer_norm_backward(prnn_dtype_t dtype, long long rows, int cols,
                                       const void* dy, long long dy_stride, const void* x,
                                       long long x_stride, const float* gamma, const float* mean,
                                       const float* rstd, void* dx, long long dx_stride,
                                       float* dgamma, float* dbeta, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!known(dtype) || rows < 0 || cols < 1) return PRNN_ERR_INVALID_ARG;
  const size_t esz = elem_size(dtype);
  if (!aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) ||
      !aligned(dbeta, 4))
    return PRNN_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dgamma && dbeta && overlaps(dgamma, 4ull * cols, dbeta, 4ull * cols))
    return PRNN_ERR_INVALID_ARG;
  if (rows == 0) {
    if (dgamma) PRNN_TRY(cudaMemsetAsync(dgamma, 0, 4ull * cols, s));
    if (dbeta) PRNN_TRY(cudaMemsetAsync(dbeta, 0, 4ull * cols, s));
    return PRNN_OK;
  }
  if (!dy || !x || !mean || !rstd || !aligned(dy, esz) || !aligned(x, esz) || !aligned(dx, esz))
    return PRNN_ERR_INVALID_ARG;
  if (rows > 1 && (x_stride < cols || dy_stride < cols || (dx && dx_stride < cols)))
    return PRNN_ERR_INVALID_ARG;
  const long long nx = row_extent(rows, cols, rows > 1 ? x_stride : cols);
  const long long ny = row_extent(rows, cols, rows > 1 ? dy_stride : cols);
  const long long nd = row_extent(rows, cols, rows > 1 ? dx_stride : cols);
  if (nx < 0 || ny < 0 || nd < 0) return PRNN_ERR_INVALID_ARG;
  size_t need = 0;
  prnn_layer_norm_workspace(rows, cols, &need);
  const bool sums = dgamma || dbeta;
  if (sums && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return PRNN_ERR_INVALID_ARG;
  struct Arr { const void* p; size_t n; };
  const Arr ins[] = {{x, nx * esz}, {dy, ny * esz}, {gamma, 4ull * cols}, {mean, 4ull * rows},
                     {rstd, 4ull * rows}};
  const Arr outs[] = {{dx, nd * esz}, {dgamma, 4ull * cols}, {dbeta, 4ull * cols},
                      {sums ? workspace : nullptr, need}};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i].p) continue;
    for (const Arr& q : ins)
      if (q.p && overlaps(outs[i].p, outs[i].n, q.p, q.n)) return PRNN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[j].p && overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return PRNN_ERR_INVALID_ARG;
  }
  LayerNormGradArgs a{dtype, rows, cols, dy, x, dy_stride, x_stride, gamma, mean, rstd,
                      dx,    dx_stride, dgamma, dbeta, static_cast<float*>(workspace)};
  return cuda_status(launch_layer_norm_grad(a, s));
}

prnn_status_t prnn_dropout_forward(prnn_dtype_t dtype, long long n, const void* x,
                                   const void* residual, void* y, double p, uint64_t seed,
                                   uint64_t offset, void* stream) {
  if (!known(dtype) || n < 0 || n > LLONG_MAX / 8 || !(p >= 0.0 && p < 1.0))
    return PRNN_ERR_INVALID_ARG;
  const double limit = std::nearbyint(p * 4294967296.0);
  if (limit >= 4294967296.0) return PRNN_ERR_INVALID_ARG;
  if (n == 0) return PRNN_OK;
  const size_t esz = elem_size(dtype);
  if (!x || !y || !aligned(x, esz) || !aligned(y, esz) || !aligned(residual, esz))
    return PRNN_ERR_INVALID_ARG;
  if (x != y && overlaps(x, n * esz, y, n * esz)) return PRNN_ERR_INVALID_ARG;
  if (residual && residual != y && overlaps(residual, n * esz, y, n * esz))
    return PRNN_ERR_INVALID_ARG;
  DropoutArgs a{dtype, n, x, residual, y, (uint32_t)limit, (float)(1.0 / (1.0 - p)), seed, offset};
  return cuda_status(launch_dropout(a, static_cast<cudaStream_t>(stream)));
}

prnn_status_t prnn_dropout_backward(prnn_dtype_t dtype, long long n, const void* dy, void* dx,
                                    double p, uint64_t seed, uint64_t offset, void* stream) {
  return prnn_dropout_forward(dtype, n, dy, nullptr, dx, p, seed, offset, stream);
}

prnn_status_t prnn_linear_attention_workspace(const prnn_linear_attention_t* a, int backward,
                                              size_t* bytes) {
  prnn_status_t why;
  if (!bytes) return PRNN_ERR_INVALID_ARG;
  if (!shape_ok(a, &why)) return why;
  *bytes = (backward ? 2 * group_bytes(a) : 0) + mix_bytes(a, backward != 0);
  return PRNN_OK;
}

prnn_status_t prnn_linear_attention_forward(const prnn_linear_attention_t* a, void* stream) {
  prnn_status_t why;
  if (!shape_ok(a, &why)) return why;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->B == 0) return PRNN_OK;
  const size_t state_bytes = sizeof(float) * (size_t)a->B * a->heads * a->dk * a->dv;
  if (!aligned(a->state, 4) || !aligned(a->state_out, 4) || !aligned(a->lens, 4))
    return PRNN_ERR_INVALID_ARG;
  if (a->state && a->state_out && a->state != a->state_out &&
      overlaps(a->state, state_bytes, a->state_out, state_bytes))
    return PRNN_ERR_INVALID_ARG;
  if (a->T == 0) {
    if (!a->state_out || a->state_out == a->state) return PRNN_OK;
    if (a->state)
      return cuda_status(cudaMemcpyAsync(a->state_out, a->state, state_bytes,
                                         cudaMemcpyDeviceToDevice, s));
    return cuda_status(cudaMemsetAsync(a->state_out, 0, state_bytes, s));
  }
  if (!a->log_decay || !aligned(a->log_decay, 4)) return PRNN_ERR_INVALID_ARG;
  const size_t esz = elem_size(a->dtype);
  const int T = a->T, B = a->B, H = a->heads, Hq = a->qk_heads;
  const Part part[] = {{a->q.data, dims_of(a->q, T, B, Hq, a->dk), false},
                       {a->k.data, dims_of(a->k, T, B, Hq, a->dk), false},
                       {a->v.data, dims_of(a->v, T, B, H, a->dv), false},
                       {a->o.data, dims_of(a->o, T, B, H, a->dv), true}};
  const prnn_seq_t* seq[] = {&a->q, &a->k, &a->v, &a->o};
  for (int i = 0; i < 4; ++i)
    if (!seq_ok(*seq[i], part[i].d, esz, part[i].out)) return PRNN_ERR_INVALID_ARG;
  if (!outputs_apart(part, 4, esz)) return PRNN_ERR_INVALID_ARG;
  if ((a->state && !clear_of(a->state, state_bytes, part, 4, esz, false)) ||
      (a->state_out && !clear_of(a->state_out, state_bytes, part, 4, esz, true)) ||
      !clear_of(a->log_decay, 4ull * H, part, 4, esz, false) ||
      (a->lens && !clear_of(a->lens, 4ull * B, part, 4, esz, false)))
    return PRNN_ERR_INVALID_ARG;
  const size_t need = mix_bytes(a, false);
  if (need && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need ||
               !clear_of(a->workspace, need, part, 4, esz, true) ||
               (a->state && overlaps(a->state, state_bytes, a->workspace, need)) ||
               (a->state_out && overlaps(a->state_out, state_bytes, a->workspace, need))))
    return PRNN_ERR_INVALID_ARG;
  if (!tables_clear(a->state_out, state_bytes, a, a->lens) || !tables_clear(a->workspace, need, a, a->lens))
    return PRNN_ERR_INVALID_ARG;
  LaArgs g{};
  LaRole& r = g.role[0];
  r.a = in(a->q, H / Hq);
  r.b = in(a->k, H / Hq);
  r.c = in(a->v, 1);
  r.out = a->o.data;
  r.ot = a->o.stride_t;
  r.ob = a->o.stride_b;
  r.oh = a->o.stride_h;
  r.d = a->dk;
  r.e = a->dv;
  r.x0 = a->state;
  r.x_end = a->state_out;
  r.lead = 1;
  r.s_intra = r.s_inter = a->scale;
  r.s_add = 1.f;
  g.roles = 1;
  g.dtype = a->dtype;
  g.T = T;
  g.B = B;
  g.H = H;
  g.log_decay = a->log_decay;
  g.lens = a->lens;
  return cuda_status(launch_mix(g, a->workspace, need, s));
}

prnn_status_t prnn_linear_attention_backward(const prnn_linear_attention_t* a, void* stream) {
  prnn_status_t why;
  if (!shape_ok(a, &why)) return why;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->B == 0) return PRNN_OK;
  const size_t state_bytes = sizeof(float) * (size_t)a->B * a->heads * a->dk * a->dv;
  if (!aligned(a->state, 4) || !aligned(a->d_state_out, 4) || !aligned(a->d_state, 4) ||
      !aligned(a->lens, 4))
    return PRNN_ERR_INVALID_ARG;
  if (a->d_state && ((a->state && overlaps(a->state, state_bytes, a->d_state, state_bytes)) ||
                     (a->d_state_out &&
                      overlaps(a->d_state_out, state_bytes, a->d_state, state_bytes))))
    return PRNN_ERR_INVALID_ARG;
  if (a->T == 0) {
    if (!a->d_state) return PRNN_OK;
    if (a->d_state_out)
      return cuda_status(cudaMemcpyAsync(a->d_state, a->d_state_out, state_bytes,
                                         cudaMemcpyDeviceToDevice, s));
    return cuda_status(cudaMemsetAsync(a->d_state, 0, state_bytes, s));
  }
  if (!a->log_decay || !aligned(a->log_decay, 4)) return PRNN_ERR_INVALID_ARG;
  const size_t esz = elem_size(a->dtype);
  const int T = a->T, B = a->B, H = a->heads, Hq = a->qk_heads, G = H / Hq;
  const prnn_seq_t* seq[] = {&a->q, &a->k, &a->v, &a->d_o, &a->d_q, &a->d_k, &a->d_v};
  const int heads[] = {Hq, Hq, H, H, Hq, Hq, H};
  const int width[] = {a->dk, a->dk, a->dv, a->dv, a->dk, a->dk, a->dv};
  Part part[7];
  int n = 0;
  for (int i = 0; i < 7; ++i) {
    const bool out = i >= 4;
    if (out && !seq[i]->data) continue;
    part[n] = {seq[i]->data, dims_of(*seq[i], T, B, heads[i], width[i]), out};
    if (!seq_ok(*seq[i], part[n].d, esz, out)) return PRNN_ERR_INVALID_ARG;
    ++n;
  }
  if (!outputs_apart(part, n, esz)) return PRNN_ERR_INVALID_ARG;
  size_t need = 0;
  prnn_linear_attention_workspace(a, 1, &need);
  if (need && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need))
    return PRNN_ERR_INVALID_ARG;
  if ((a->state && !clear_of(a->state, state_bytes, part, n, esz, false)) ||
      (a->d_state_out && !clear_of(a->d_state_out, state_bytes, part, n, esz, false)) ||
      (a->d_state && !clear_of(a->d_state, state_bytes, part, n, esz, true)) ||
      (need && !clear_of(a->workspace, need, part, n, esz, true)) ||
      !clear_of(a->log_decay, 4ull * H, part, n, esz, false) ||
      (a->lens && !clear_of(a->lens, 4ull * B, part, n, esz, false)))
    return PRNN_ERR_INVALID_ARG;
  if (need)
    for (const float* p : {a->state, a->d_state_out, static_cast<const float*>(a->d_state)})
      if (p && overlaps(p, state_bytes, a->workspace, need)) return PRNN_ERR_INVALID_ARG;
  if (!tables_clear(a->d_state, state_bytes, a, a->lens) || !tables_clear(a->workspace, need, a, a->lens))
    return PRNN_ERR_INVALID_ARG;

  LaArgs g{};
  g.dtype = a->dtype;
  g.T = T;
  g.B = B;
  g.H = H;
  g.log_decay = a->log_decay;
  g.lens = a->lens;
  float* part_q = static_cast<float*>(a->workspace);
  float* part_k = part_q + group_bytes(a) / sizeof(float);
  // heads that share a query and key head leave fp32 parts, summed afterwards
  auto out_to = [&](LaRole& r, const prnn_seq_t& x, float* parts) {
    if (G > 1 && parts) {
      r.out = parts;
      r.out_f32 = 1;
      r.ot = (long long)B * H * a->dk;
      r.ob = (long long)H * a->dk;
      r.oh = a->dk;
    } else {
      r.out = x.data;
      r.ot = x.stride_t;
      r.ob = x.stride_b;
      r.oh = x.stride_h;
    }
  };
  if (a->d_q.data) {
    LaRole& r = g.role[g.roles++];
    r.a = in(a->d_o, 1);
    r.b = in(a->v, 1);
    r.c = in(a->k, G);
    out_to(r, a->d_q, part_q);
    r.d = a->dv;
    r.e = a->dk;
    r.x0 = a->state;
    r.x_t = 1;
    r.lead = 1;
    r.s_intra = r.s_inter = a->scale;
    r.s_add = 1.f;
  }
  if (a->d_k.data) {
    LaRole& r = g.role[g.roles++];
    r.a = in(a->v, 1);
    r.b = in(a->d_o, 1);
    r.c = in(a->q, G);
    out_to(r, a->d_k, part_k);
    r.d = a->dv;
    r.e = a->dk;
    r.x0 = a->d_state_out;
    r.x_t = 1;
    r.rev = 1;
    r.s_intra = r.s_add = a->scale;
    r.s_inter = 1.f;
  }
  if (a->d_v.data || a->d_state) {
    LaRole& r = g.role[g.roles++];
    r.a = in(a->k, G);
    r.b = in(a->q, G);
    r.c = in(a->d_o, 1);
    out_to(r, a->d_v, nullptr);
    r.d = a->dk;
    r.e = a->dv;
    r.x0 = a->d_state_out;
    r.x_end = a->d_state;
    r.rev = 1;
    r.s_intra = r.s_add = a->scale;
    r.s_inter = 1.f;
  }
  PRNN_TRY(launch_mix(g, static_cast<char*>(a->workspace) + 2 * group_bytes(a),
                      need - 2 * group_bytes(a), s));
  if (G > 1) {
    const prnn_seq_t* out[] = {&a->d_q, &a->d_k};
    float* parts[] = {part_q, part_k};
    for (int i = 0; i < 2; ++i) {
      if (!out[i]->data) continue;
      LaReduceArgs r{a->dtype, parts[i], out[i]->data, out[i]->stride_t, out[i]->stride_b,
                     out[i]->stride_h, T, B, H, G, a->dk};
      PRNN_TRY(launch_la_reduce(r, s));
    }
  }
  return PRNN_OK;
}

prnn_status_t prnn_linear_attention_step(const prnn_linear_attention_t* a, float* state_pool,
                                         int n_slots, const int32_t* slots, void* stream) {
  prnn_status_t why;
  if (!shape_ok(a, &why)) return why;
  if (n_slots < 0) return PRNN_ERR_INVALID_ARG;
  if (a->B == 0) return PRNN_OK;
  if (!state_pool || !a->log_decay || !aligned(state_pool, 4) || !aligned(a->log_decay, 4) ||
      !aligned(slots, 4) || (!slots && n_slots < a->B))
    return PRNN_ERR_INVALID_ARG;
  const size_t esz = elem_size(a->dtype);
  const int B = a->B, H = a->heads, Hq = a->qk_heads;
  const size_t pool_bytes = sizeof(float) * (size_t)n_slots * H * a->dk * a->dv;
  prnn_seq_t sq[4] = {a->q, a->k, a->v, a->o};
  const int heads[] = {Hq, Hq, H, H}, width[] = {a->dk, a->dk, a->dv, a->dv};
  Part part[4];
  for (int i = 0; i < 4; ++i) {
    sq[i].stride_t = 0;
    part[i] = {sq[i].data, dims_of(sq[i], 1, B, heads[i], width[i]), i == 3};
    if (!seq_ok(sq[i], part[i].d, esz, part[i].out)) return PRNN_ERR_INVALID_ARG;
  }
  if (!outputs_apart(part, 4, esz) || !clear_of(state_pool, pool_bytes, part, 4, esz, true) ||
      !clear_of(a->log_decay, 4ull * H, part, 4, esz, false) ||
      (slots && !clear_of(slots, 4ull * B, part, 4, esz, false)) || !tables_clear(state_pool, pool_bytes, a, slots))
    return PRNN_ERR_INVALID_ARG;
  LaStepArgs r{};
  r.dtype = a->dtype;
  r.B = B;
  r.H = H;
  r.dk = a->dk;
  r.dv = a->dv;
  r.q = in(a->q, H / Hq);
  r.k = in(a->k, H / Hq);
  r.v = in(a->v, 1);
  r.o = a->o.data;
  r.ob = a->o.stride_b;
  r.oh = a->o.stride_h;
  r.log_decay = a->log_decay;
  r.state = state_pool;
  r.n_slots = n_slots;
  r.slots = slots;
  r.scale = a->scale;
  return cuda_status(launch_la_step(r, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
