// gated_delta_tc_grad.cu -- the chunks' gradients of the gated delta rule on the 5th-generation tensor cores: what the
// walk over the states' gradients needs beforehand, and what follows from it.  The algebra and the rounding are in
// gated_delta_tc.cuh.
//
// Two operands in three parts and a piece of a third fill an SM's shared memory, so one block of 16 warps works through its
// steps one behind another: latency bounds both kernels (T = 2048, 4 sequences of 16 heads of 128 x 128 bf16: 98 and 351 us,
// 0.25 instructions a cycle and scheduler, DRAM at a fifth of its rate).  32 warps took 466 us, for their registers.
#include "gated_delta_tc.cuh"

namespace prnn {
namespace gd {
namespace {

constexpr int kThreads = 512;
// Two operands of [128][128] in three parts, and a third by pieces of 64 columns and as many tokens as fit.
constexpr uint32_t kMatrix = kP * 2 * kTile, kOne = 0, kTwo = kMatrix, kThree = 2 * kMatrix, kPiece = 24 * 1024,
                   kTab = kThree + kPiece;
struct Tab {
  Gates gates;
  float rows[4][3][C];   // per quarter of the columns: q . dq, v . dv, and dbeta's sum
  float leaves[kThreads / 32];
  uint64_t bar;
  uint32_t tmem;
};
static_assert(kTab + sizeof(Tab) <= 227 * 1024, "shared memory");

// A product over the chunk's tokens with a data tensor x (its rows tokens, MN-major) as the right operand,
// piece by piece; `issue` gets the piece's tile of columns, its first step of 16 tokens, the operand, its steps
// and whether it adds to what earlier tokens left.  The first piece has been requested by `first`.
template <typename T>
struct Pieces {
  static constexpr int DP = kData<T>, ROWS = DP * kTile <= kPiece ? C : C / 2;
  DataRows<T, ROWS, 1, kThreads> rows;
  const T* x;
  long long st;
  int n, d, tiles;
  __device__ __forceinline__ void fetch(int ct, int r0) { rows.fetch(x, st, r0, n, ct * 64, d, 1); }
  __device__ __forceinline__ void first(const T* x_, long long st_, int n_, int d_, int tiles_) {
    x = x_;
    st = st_;
    n = n_;
    d = d_;
    tiles = tiles_;
    fetch(0, 0);
  }
  template <typename F>
  __device__ __forceinline__ void multiply(Steps& steps, unsigned char* smem, F&& issue) {
    int ct = 0, r0 = 0;
    while (ct < tiles) {
      rows.template place<DP>(smem + kThree, ROWS * 128, ROWS * 128);
      steps.run([&] {
        issue(ct, r0 / 16, mn_major(smem_u32(smem) + kThree, ROWS * 128, ROWS * 128), ROWS / 16, r0 > 0);
      });
      r0 += ROWS;
      if (r0 >= n || r0 >= C) {
        r0 = 0;
        ++ct;
      }
      if (ct < tiles) fetch(ct, r0);
      steps.wait();
    }
  }
};
// The left operand of such a product from its step of 16 tokens on.
__device__ __forceinline__ Operand from_step(Operand o, int k) {
  o.desc += o.tile ? (k >> 2) * o.tile + (k & 3) * 2 : k * 128;
  return o;
}

// ---- before the walk backwards: X0 = ((Q K^T) o D)^T dO, Z0 = (e^G Q)^T dO, dO times scale -------------------
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) gd_before_reverse_kernel(const __grid_constant__ Args g) {
  constexpr int DP = kData<T>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Tab& tab = *reinterpret_cast<Tab*>(smem + kTab);
  const GdArgs& a = g.a;
  const Place p = place_of(g, blockIdx.x);
  if (p.n == 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = (warp & 3) * 32 + lane, quarter = warp >> 2;
  const T *q = rows_of<T>(a.q, p.t0, p.b, p.hq), *k = rows_of<T>(a.k, p.t0, p.b, p.hq),
          *d_o = rows_of<T>(a.d_o, p.t0, p.b, p.h);
  DataRows<T, C, 2, kThreads> qs, ks;
  qs.fetch(q, a.q.st, 0, p.n, 0, a.dk, g.dkt);
  ks.fetch(k, a.k.st, 0, p.n, 0, a.dk, g.dkt);
  if (!begin(&tab.bar, &tab.tmem, 512, smem, g.status)) return;
  Steps steps{&tab.bar};
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16), base = smem_u32(smem);
  copy_gates<kThreads>(tab.gates, g.gates + p.at);
  const int rows = 64 * g.dkt, cols = 64 * g.dvt;
  const uint32_t part = g.dkt * kTile;
  qs.template place<DP>(smem + kOne, part, kTile);
  ks.template place<DP>(smem + kTwo, part, kTile);
  steps.run([&] {
    product<DP, DP>(tmem, k_major(base + kOne, part, kTile), k_major(base + kTwo, part, kTile), (a.dk + 15) / 16,
                    id_of(128, false, false), false);
  });
  Pieces<T> dos;
  dos.first(d_o, a.d_o.st, p.n, a.dv, g.dvt);
  steps.wait();
  if (tid < C) tab.rows[0][0][tid] = a.scale * tab.gates.up[tid];
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    const int c0 = quarter * 32 + x * 16;
    float2 v[8];
    if (quarter <= (warp & 3)) read16(mine + c0, v);
    decayed<false>(v, row, c0, tab.gates);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], both(a.scale));
    put16<kP>(smem + kTwo, 2 * kTile, row, c0, v);
  }
  __syncthreads();
  qs.template place<kP>(smem + kOne, part, kTile, tab.rows[0][0]);
  const Operand P = mn_major(base + kTwo, 2 * kTile, kTile), Q = mn_major(base + kOne, part, kTile);
  dos.multiply(steps, smem, [&](int ct, int k0, const Operand& right, int n, bool add) {
    product<kP, DP>(tmem + 128 + 64 * ct, from_step(P, k0), right, n, id_of(64, true, true), add);
    product<kP, DP>(tmem + 256 + 64 * ct, from_step(Q, k0), right, n, id_of(64, true, true), add);
  });
  float *X = g.X + p.at * C * cols, *Z0 = g.Z0 + p.at * rows * cols;
#pragma unroll 1
  for (int x = 0; x < g.dvt; ++x) {
    const int c0 = (quarter * g.dvt + x) * 16;
    float2 v[8];
    read16(mine + 128 + c0, v);
    store_quads(X, C, row, c0, v);
    read16(mine + 256 + c0, v);
    if (row < rows) store_quads(Z0, rows, row, c0, v);
  }
  finish(tmem, 512, steps.ok, g.status);
}

// ---- the gradients of a chunk ----------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) gd_gradients_kernel(const __grid_constant__ Args g) {
  constexpr int DP = kData<T>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Tab& tab = *reinterpret_cast<Tab*>(smem + kTab);
  const GdArgs& a = g.a;
  const Place p = place_of(g, blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = (warp & 3) * 32 + lane, quarter = warp >> 2;
  // Where this head's rows of a gradient go: the tensor itself, or fp32 parts that are joined later.
  struct Rows {
    T* out;
    float* part;
    long long st, part_st;
    int d;
    __device__ __forceinline__ void store(long long t, int c0, const float2 (&v)[8]) const {
      if (part) store16<float>(part + t * part_st + c0, d - c0, v);
      else if (out) store16<T>(out + t * st + c0, d - c0, v);
    }
    __device__ __forceinline__ void zero(long long t, int c) const {
      if (part) part[t * part_st + c] = 0.f;
      else if (out) out[t * st + c] = from_f32<T>(0.f);
    }
  };
  auto rows_to = [&](void* out, float* part, long long st, long long sb, long long sh, int d) {
    return Rows{out ? static_cast<T*>(out) + p.b * sb + p.h * sh : nullptr,
                part ? part + ((long long)p.b * a.H + p.h) * d : nullptr, st, (long long)a.B * a.H * d, d};
  };
  const Rows dq = rows_to(a.dq_out, a.dq_part, a.dqt, a.dqb, a.dqh, a.dkp),
             dk = rows_to(a.dk_out, a.dk_part, a.dkt, a.dkb, a.dkh, a.dkp),
             dv = rows_to(a.dv_out, a.dv_part, a.dvt, a.dvb, a.dvh, a.dvp);
  const int live = (int)(a.T - p.t0 < C ? a.T - p.t0 : C);  // rows of the tensors
  for (int r = p.n; r < live; ++r) {                        // zeros past the length
    if (tid < a.dkp) {
      dq.zero(p.t0 + r, tid);
      dk.zero(p.t0 + r, tid);
    }
    if (tid < a.dvp) dv.zero(p.t0 + r, tid);
    if (tid == 0) {
      if (a.dg) a.dg[(p.t0 + r) * a.dgt + p.b * a.dgb + p.h * a.dgh] = 0.f;
      if (a.dbeta) a.dbeta[(p.t0 + r) * a.dbt + p.b * a.dbb + p.h * a.dbh] = 0.f;
    }
  }
  if (p.n == 0) return;
  if (!begin(&tab.bar, &tab.tmem, 512, smem, g.status)) return;
  Steps steps{&tab.bar};
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16), base = smem_u32(smem);
  const uint32_t D0 = 0, D1 = 128, D2 = 256, D3 = 384;
  copy_gates<kThreads>(tab.gates, g.gates + p.at);
  __syncthreads();
  const int rows = 64 * g.dkt, cols = 64 * g.dvt;
  const uint32_t kpart = g.dkt * kTile, vpart = g.dvt * kTile;
  const float *E = g.E + p.at * C * cols, *X = g.X + p.at * C * cols, *S = g.S + p.slot * rows * cols,
              *R = g.R + p.at * rows * cols, *inv = g.inv + p.at * C * C;
  const T *q = rows_of<T>(a.q, p.t0, p.b, p.hq), *k = rows_of<T>(a.k, p.t0, p.b, p.hq),
          *v = rows_of<T>(a.v, p.t0, p.b, p.h), *d_o = rows_of<T>(a.d_o, p.t0, p.b, p.h);
  if (tid == 0) {  // what later steps load
    ask_l2(E, C * cols * 4);
    ask_l2(S, rows * cols * 4);
    ask_l2(R, rows * cols * 4);
  }
  const float up = tab.gates.up[row], down = tab.gates.down[row], beta = tab.gates.beta[row];
  const bool mine_live = row < p.n;
  DataRows<T, C, 2, kThreads> data;
  Pieces<T> pieces;
  auto quads = [&](uint32_t where, const float* m, int rows_, int tiles, const float* scale) {
    load_quads<kP, kThreads>(smem + where, tiles * kTile, m, rows_, tiles, scale);
  };
  // this row's 16 values at columns c0 of a data tensor's row times f, summed
  auto dot_row = [&](const Pack<T, 8> (&x)[2], const float2 (&f)[8]) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 y[4];
      pairs_of<T>(x[j], y);
#pragma unroll
      for (int k = 0; k < 4; ++k) s = fmaf(y[k].x, f[4 * j + k].x, fmaf(y[k].y, f[4 * j + k].y, s));
    }
    return s;
  };
  auto ask_row = [&](Pack<T, 8> (&x)[2], const T* from, int c0, int d) {
#pragma unroll
    for (int j = 0; j < 2; ++j) x[j] = mine_live && c0 + 8 * j < d ? get8<T>(from + c0 + 8 * j) : zeros8<T>();
  };

  // dV = Tt^T (beta X)
  quads(kOne, inv, C, 2, nullptr);
  quads(kTwo, X, C, g.dvt, tab.gates.beta);
  steps.run([&] {
    product<kP, kP>(tmem + D0, mn_major(base + kOne, 2 * kTile, kTile), mn_major(base + kTwo, vpart, kTile), 8,
                    id_of(cols, true, true), false);
  });
  // dbeta_i = e_i . du_i, du_i = dv_i / beta_i = x_i - sum_{j > i} M_ji dv_j.  The quotient keeps its bits however small
  // beta is (dv_i is beta_i times sums without it); the difference cancels where keys repeat, and stands for beta = 0.
  const bool tiny = !(fabsf(beta) > 1e-20f);
  const bool any_tiny = __syncthreads_or(tiny && mine_live);
  float es = 0.f;  // e . x or e . dv
  if (any_tiny)
    for (int c = quarter * 16 * g.dvt; c < (quarter + 1) * 16 * g.dvt; c += 4) {
      const size_t i = (size_t)(c / 4) * C + row;
      const float4 e = reinterpret_cast<const float4*>(E)[i], x = reinterpret_cast<const float4*>(X)[i];
      es = fmaf(e.x, x.x, fmaf(e.y, x.y, fmaf(e.z, x.z, fmaf(e.w, x.w, es))));
    }
  steps.wait();
  {
    float s = 0.f, ev = 0.f;
#pragma unroll 1
    for (int x = 0; x < g.dvt; ++x) {
      const int c0 = (quarter * g.dvt + x) * 16;
      float2 f[8];
      Pack<T, 8> vs[2];
      ask_row(vs, v + row * a.v.st, c0, a.dv);
      read16(mine + D0 + c0, f);
      if (mine_live) {
        s += dot_row(vs, f);
        dv.store(p.t0 + row, c0, f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 e = reinterpret_cast<const float4*>(E)[(size_t)(c0 / 4 + i) * C + row];
        ev = fmaf(e.x, f[2 * i].x, fmaf(e.y, f[2 * i].y, fmaf(e.z, f[2 * i + 1].x, fmaf(e.w, f[2 * i + 1].y, ev))));
      }
      put16<kP>(smem + kTwo, vpart, row, c0, f);
    }
    tab.rows[quarter][1][row] = s;
    if (!tiny) es = ev / beta;
  }
  // dV E^T, and where a beta is 0, E dV^T and K K^T
  quads(kOne, E, C, g.dvt, nullptr);
  const Operand one_v = k_major(base + kOne, vpart, kTile), two_v = k_major(base + kTwo, vpart, kTile);
  const int vsteps = (a.dv + 15) / 16, ksteps = (a.dk + 15) / 16;
  steps.run([&] {
    product<kP, kP>(tmem + D0, two_v, one_v, vsteps, id_of(128, false, false), false);
    if (any_tiny) product<kP, kP>(tmem + D1, one_v, two_v, vsteps, id_of(128, false, false), false);
  });
  pieces.first(k, a.k.st, p.n, a.dk, g.dkt);
  steps.wait();
  if (any_tiny) {  // es -= sum over j > i of (k_i . k_j) D_ji (e_i . dv_j)
    data.fetch(k, a.k.st, 0, p.n, 0, a.dk, g.dkt);
    data.template place<DP>(smem + kOne, kpart, kTile);
    steps.run([&] {
      const Operand K = k_major(base + kOne, kpart, kTile);
      product<DP, DP>(tmem + D2, K, K, ksteps, id_of(128, false, false), false);
    });
    steps.wait();
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      const int c0 = quarter * 32 + x * 16;
      if (quarter < (warp & 3)) continue;
      float2 y[8], kk[8];
      read16(mine + D1 + c0, y);
      read16(mine + D2 + c0, kk);
      const float2 here = tab.gates.sum[row];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float f = at_of16(kk, i) * at_of16(y, i) * decay_between(tab.gates.sum[c0 + i], here);
        es -= tiny && c0 + i > row ? f : 0.f;
      }
    }
  }
  tab.rows[quarter][2][row] = es;
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {  // -Y as the next left operand
    const int c0 = quarter * 32 + x * 16;
    float2 y[8];
    if (quarter <= (warp & 3)) read16(mine + D0 + c0, y);
    decayed<true>(y, row, c0, tab.gates);
    times16(y, tab.gates.beta + c0);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = mul2(y[i], both(-1.f));
    put16<kP>(smem + kOne, 2 * kTile, row, c0, y);
  }
  before_sync();
  __syncthreads();
  after_sync();
  // D3 = -(Y + Y^T) K, Y in both majors
  const Operand one_t = k_major(base + kOne, 2 * kTile, kTile), one_tt = mn_major(base + kOne, 2 * kTile, kTile);
  pieces.multiply(steps, smem, [&](int ct, int k0, const Operand& right, int n, bool add) {
    product<kP, DP>(tmem + D3 + 64 * ct, from_step(one_t, k0), right, n, id_of(64, false, true), add);
    product<kP, DP>(tmem + D3 + 64 * ct, from_step(one_tt, k0), right, n, id_of(64, true, true), true);
  });
  // D0 = dV S0^T
  quads(kOne, S, rows, g.dvt, nullptr);
  steps.run([&] { product<kP, kP>(tmem + D0, two_v, one_v, vsteps, id_of(rows, false, false), false); });
  data.fetch(d_o, a.d_o.st, 0, p.n, 0, a.dv, g.dvt);
  steps.wait();
  // D1 = dO S0^T
  data.template place<DP>(smem + kTwo, vpart, kTile);
  steps.run([&] { product<DP, kP>(tmem + D1, two_v, one_v, vsteps, id_of(rows, false, false), false); });
  steps.wait();
  // D2 = dO U^T
  quads(kOne, E, C, g.dvt, tab.gates.beta);
  steps.run([&] { product<DP, kP>(tmem + D2, two_v, one_v, vsteps, id_of(128, false, false), false); });
  pieces.first(k, a.k.st, p.n, a.dk, g.dkt);
  steps.wait();
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    const int c0 = quarter * 32 + x * 16;
    float2 f[8];
    if (quarter <= (warp & 3)) read16(mine + D2 + c0, f);
    decayed<false>(f, row, c0, tab.gates);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = mul2(f[i], both(a.scale));
    put16<kP>(smem + kTwo, 2 * kTile, row, c0, f);
  }
  before_sync();
  __syncthreads();
  after_sync();
  // D2 = Z K
  const Operand two_t = k_major(base + kTwo, 2 * kTile, kTile), two_tt = mn_major(base + kTwo, 2 * kTile, kTile);
  pieces.multiply(steps, smem, [&](int ct, int k0, const Operand& right, int n, bool add) {
    product<kP, DP>(tmem + D2 + 64 * ct, from_step(two_t, k0), right, n, id_of(64, false, true), add);
  });
  pieces.first(q, a.q.st, p.n, a.dk, g.dkt);
  {
    float s = 0.f;
    const float f0 = a.scale * up;
#pragma unroll 1
    for (int x = 0; x < g.dkt; ++x) {
      const int c0 = (quarter * g.dkt + x) * 16;
      float2 f[8], h[8];
      Pack<T, 8> qs[2];
      ask_row(qs, q + row * a.q.st, c0, a.dk);
      read16(mine + D1 + c0, f);
      read16(mine + D2 + c0, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fma2(both(f0), f[i], h[i]);
      if (mine_live) {
        s += dot_row(qs, f);
        dq.store(p.t0 + row, c0, f);
      }
    }
    tab.rows[quarter][0][row] = s;
  }
  before_sync();
  __syncthreads();
  after_sync();
  // D2 = Z^T Q
  pieces.multiply(steps, smem, [&](int ct, int k0, const Operand& right, int n, bool add) {
    product<kP, DP>(tmem + D2 + 64 * ct, from_step(two_tt, k0), right, n, id_of(64, true, true), add);
  });
  // D1 = U R^T
  quads(kTwo, R, rows, g.dvt, nullptr);
  steps.run([&] { product<kP, kP>(tmem + D1, one_v, two_v, vsteps, id_of(rows, false, false), false); });
  // <S, R> where the chunk ends
  float leave = 0.f;
  for (int i = tid; i < rows * ((a.dv + 3) / 4); i += kThreads) {  // columns behind dv may never have been written
    const float4 s = reinterpret_cast<const float4*>(S + rows * cols)[i], r = reinterpret_cast<const float4*>(R)[i];
    leave = fmaf(s.x, r.x, fmaf(s.y, r.y, fmaf(s.z, r.z, fmaf(s.w, r.w, leave))));
  }
  leave = warp_sum(leave);
  if (lane == 0) tab.leaves[warp] = leave;
  steps.wait();
#pragma unroll 1
  for (int x = 0; x < g.dkt; ++x) {
    const int c0 = (quarter * g.dkt + x) * 16;
    float2 f[8], h[8];
    read16(mine + D3 + c0, f);
    read16(mine + D2 + c0, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = add2(f[i], h[i]);
    read16(mine + D0 + c0, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fma2(both(-up), h[i], f[i]);
    read16(mine + D1 + c0, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fma2(both(down), h[i], f[i]);
    if (mine_live) dk.store(p.t0 + row, c0, f);
  }
  __syncthreads();
  if (warp == 0) {  // the gates: a lane has 4 tokens, summed from the chunk's end
    auto all = [&](int what, int r) {
      return (tab.rows[0][what][r] + tab.rows[1][what][r]) + (tab.rows[2][what][r] + tab.rows[3][what][r]);
    };
    float base_ = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) base_ += tab.leaves[i];
    float s[4], run = 0.f;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const int r = lane * 4 + i;
      s[i] = run += r < p.n ? all(0, r) - all(1, r) : 0.f;
    }
    float after = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_down_sync(0xffffffffu, after, o);
      if (lane + o < 32) after += x;
    }
    after = __shfl_down_sync(0xffffffffu, after, 1);
    if (lane == 31) after = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = lane * 4 + i;
      if (r >= p.n) continue;
      if (a.dg) a.dg[(p.t0 + r) * a.dgt + p.b * a.dgb + p.h * a.dgh] = s[i] + after + base_;
      if (a.dbeta)
        a.dbeta[(p.t0 + r) * a.dbt + p.b * a.dbb + p.h * a.dbh] = all(2, r);
    }
  }
  finish(tmem, 512, steps.ok, g.status);
}

}  // namespace

cudaError_t launch_before_reverse(const Args& g, cudaStream_t s) {
  PRNN_BY_DTYPE(g.a.dtype, T, {
    constexpr uint32_t smem = kTab + sizeof(Tab);
    const cudaError_t e = cudaFuncSetAttribute(gd_before_reverse_kernel<T>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    gd_before_reverse_kernel<T><<<(unsigned)(g.nbh * g.chunks), kThreads, smem, s>>>(g);
  });
  return cudaGetLastError();
}

cudaError_t launch_gradients(const Args& g, cudaStream_t s) {
  const GdArgs& a = g.a;
  PRNN_BY_DTYPE(a.dtype, T, {
    constexpr uint32_t smem = kTab + sizeof(Tab);
    const cudaError_t e = cudaFuncSetAttribute(gd_gradients_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem);
    if (e != cudaSuccess) return e;
    gd_gradients_kernel<T><<<(unsigned)(g.nbh * g.chunks), kThreads, smem, s>>>(g);
  });
  return cudaGetLastError();
}

}  // namespace gd
}  // namespace prnn
