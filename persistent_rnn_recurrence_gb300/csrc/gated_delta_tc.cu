// gated_delta_tc.cu -- the gated delta rule's forward pass in chunks on the 5th-generation tensor cores, and the plan of
// its backward pass.  The algebra and the rounding are in gated_delta_tc.cuh.
#include <algorithm>

#include "gated_delta_tc.cuh"

namespace prnn {
namespace gd {
namespace {

// ---- before the states: gates, Tt, Tt V, W, for a chunk of a head per block ------------------------------
//
// Tt, the inverse of a unit lower triangular matrix, is made in fp32: the four diagonal blocks of 32 by
// substitution, a column per lane, then the blocks below by T_ij = -T_ii sum_m A_im T_mj, diagonal by diagonal.
constexpr int kLd = 132;  // floats of a row: 16-byte aligned, rows of a quad of banks apart
struct PrepTab {
  Gates gates;
  double part[4];
  uint64_t bar;
  uint32_t tmem;
};
constexpr uint32_t kPrepRight = 96 * 1024, kPrepTab = 192 * 1024;
static_assert(2 * C * kLd * sizeof(float) <= kPrepTab && kPrepTab + sizeof(PrepTab) <= 227 * 1024, "shared memory");

// A's and T's blocks of 32: block (i, j) of T <- -T_ii (sum_{m=j}^{i-1} A_im T_mj), the sum kept in T's unused block
// (j, i).  Q threads share a block, X x W values each.
template <int GAP>
__device__ __forceinline__ void lower_blocks(const float* A, float* T) {
  constexpr int BLOCKS = 4 - GAP, Q = GAP == 1 ? 128 : (GAP == 2 ? 256 : 512), W = GAP == 3 ? 1 : 2, X = 1024 / Q / W;
  const int j = threadIdx.x / Q, q = threadIdx.x % Q, i = j + GAP;
  const int r = q / (32 / W) * X, c = q % (32 / W) * W;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (j < BLOCKS) {
      float s[X][W];
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int y = 0; y < W; ++y) s[x][y] = 0.f;
      // pass 0: A[i][j .. i-1] T[j .. i-1][j]; pass 1: T[i][i] times that
      const float* left = pass == 0 ? A + (32 * i + r) * kLd + 32 * j : T + (32 * i + r) * kLd + 32 * i;
      const float* right = pass == 0 ? T + 32 * j * kLd + 32 * j + c : T + 32 * j * kLd + 32 * i + c;
      const int depth = pass == 0 ? 32 * GAP : 32;
#pragma unroll 2
      for (int m = 0; m < depth; m += 4) {
        float4 l[X];
        Pack<float, W> f[4];
#pragma unroll
        for (int x = 0; x < X; ++x) l[x] = *reinterpret_cast<const float4*>(left + x * kLd + m);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = load_pack<float, W>(right + (m + k) * kLd);
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int y = 0; y < W; ++y)
            s[x][y] = fmaf(l[x].w, f[3].v[y], fmaf(l[x].z, f[2].v[y], fmaf(l[x].y, f[1].v[y],
                                                                        fmaf(l[x].x, f[0].v[y], s[x][y]))));
      }
      float* to = pass == 0 ? T + (32 * j + r) * kLd + 32 * i + c : T + (32 * i + r) * kLd + 32 * j + c;
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int y = 0; y < W; ++y) to[x * kLd + y] = pass == 0 ? s[x][y] : -s[x][y];
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

constexpr int kPrepThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kPrepThreads, 1) gd_prepare_kernel(const __grid_constant__ Args g, int keep_inverse) {
  constexpr int DP = kData<T>, NT = kPrepThreads;
  extern __shared__ __align__(1024) unsigned char smem[];
  PrepTab& tab = *reinterpret_cast<PrepTab*>(smem + kPrepTab);
  const GdArgs& a = g.a;
  const Place p = place_of(g);
  if (p.n == 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = (warp & 3) * 32 + lane, quarter = warp >> 2;
  const T *k = rows_of<T>(a.k, p.t0, p.b, p.hq), *v = rows_of<T>(a.v, p.t0, p.b, p.h);
  DataRows<T, C, 2, NT> rows;
  rows.fetch(k, a.k.st, 0, p.n, 0, a.dk, g.dkt, g.vec);
  if (!begin(&tab.bar, &tab.tmem, 256, smem, g.status)) return;
  Steps steps{&tab.bar};
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16), base = smem_u32(smem);
  const uint32_t part = g.dkt * kTile, vpart = g.dvt * kTile;
  double G = 0;
  if (tid < C) {
    if (tid < p.n) {
      const long long t = p.t0 + tid;
      float x = a.g[t * a.gt + p.b * a.gb + p.h * a.gh];
      if (x < -1000.f) x = -1000.f;
      G = x * 1.4426950408889634;
      tab.gates.beta[tid] = a.beta[t * a.bt + p.b * a.bb + p.h * a.bh];
    } else {
      tab.gates.beta[tid] = 0.f;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, G, o);
      if (lane >= o) G += x;
    }
    if (lane == 31) tab.part[warp] = G;
  }
  rows.template place<DP>(smem, part, kTile);
  __syncthreads();
  if (tid < C) {
    double all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < warp) G += tab.part[w];
      all += tab.part[w];
    }
    const float hi = (float)G;
    tab.gates.hi[tid] = hi;
    tab.gates.lo[tid] = hi == hi ? (float)(G - hi) : hi;
    tab.gates.up[tid] = exp2f(hi);
    tab.gates.down[tid] = exp2f((float)(all - G));
  }
  const Operand K = k_major(base, part, kTile);
  steps.run([&] { product<DP, DP>(tmem, K, K, (a.dk + 15) / 16, id_of(128, false, false), false); });
  if (tid == 0) {  // the walk's copy of K
    for (int ct = 0; ct < g.dkt; ++ct)
      for (int q = 0; q < DP; ++q)
        bulk_store(g.kimg + ((p.at * g.dkt + ct) * DP + q) * kTile, base + q * part + ct * kTile, kTile);
    bulk_commit();
  }
  {
    const float* from = reinterpret_cast<const float*>(&tab.gates);
    float* to = reinterpret_cast<float*>(g.gates + p.at);
    for (int i = tid; i < (int)(sizeof(Gates) / 4); i += NT) to[i] = from[i];
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  steps.wait();
  __syncthreads();  // K's place may be written again
  float* A = reinterpret_cast<float*>(smem);
  float* inv = A + C * kLd;
  {  // A_ij = (k_i . k_j) D_ij beta_j below the diagonal
    const float hi = tab.gates.hi[row], lo = tab.gates.lo[row];
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      const int c0 = quarter * 32 + q * 16;
      float2 x[8];
      read16(mine + c0, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = c0 + 2 * i;
        x[i].x = j < row ? x[i].x * decay_between(hi, lo, tab.gates.hi[j], tab.gates.lo[j]) * tab.gates.beta[j] : 0.f;
        x[i].y = j + 1 < row
                     ? x[i].y * decay_between(hi, lo, tab.gates.hi[j + 1], tab.gates.lo[j + 1]) * tab.gates.beta[j + 1]
                     : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(A + row * kLd + c0 + 4 * i) =
            make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
    }
  }
  before_sync();
  __syncthreads();
  if (warp < 4) {
    float x[32];
    const float* D = A + 32 * warp * kLd + 32 * warp;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      float s[4] = {r == lane ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < r; m += 4) {
        const float4 l = *reinterpret_cast<const float4*>(D + r * kLd + m);
        s[0] = fmaf(-l.x, x[m], s[0]);
        if (m + 1 < r) s[1] = fmaf(-l.y, x[m + 1], s[1]);
        if (m + 2 < r) s[2] = fmaf(-l.z, x[m + 2], s[2]);
        if (m + 3 < r) s[3] = fmaf(-l.w, x[m + 3], s[3]);
      }
      x[r] = (s[0] + s[1]) + (s[2] + s[3]);
      inv[(32 * warp + r) * kLd + 32 * warp + lane] = x[r];
    }
  }
  __syncthreads();
  lower_blocks<1>(A, inv);
  lower_blocks<2>(A, inv);
  rows.fetch(v, a.v.st, 0, p.n, 0, a.dv, g.dvt, g.vec);
  lower_blocks<3>(A, inv);
  {  // Tt as parts, in the place of A and of itself
    float2 x[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const int c = quarter * 32 + q * 16 + 2 * i;
        const float4 f = *reinterpret_cast<const float4*>(inv + row * kLd + c);
        x[q][i] = make_float2(c <= row ? f.x : 0.f, c + 1 <= row ? f.y : 0.f);
        x[q][i + 1] = make_float2(c + 2 <= row ? f.z : 0.f, c + 3 <= row ? f.w : 0.f);
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c0 = quarter * 32 + q * 16;
      put16<kP>(smem, 2 * kTile, row, c0, x[q]);
      if (keep_inverse) store_quads(g.inv + p.at * C * C, C, row, c0, x[q]);
    }
  }
  const Operand Tt = k_major(base, 2 * kTile, kTile);
  rows.template place<DP>(smem + kPrepRight, vpart, kTile);
  steps.run([&] {
    product<kP, DP>(tmem, Tt, mn_major(base + kPrepRight, vpart, kTile), 8, id_of(64 * g.dvt, false, true), false);
  });
  rows.fetch(k, a.k.st, 0, p.n, 0, a.dk, g.dkt, g.vec);
  steps.wait();
  rows.template place<kP>(smem + kPrepRight, part, kTile, tab.gates.up);
  steps.run([&] {
    product<kP, kP>(tmem + 128, Tt, mn_major(base + kPrepRight, part, kTile), 8, id_of(64 * g.dkt, false, true), false);
  });
  float* E = g.E + p.at * C * 64 * g.dvt;
#pragma unroll 1
  for (int q = 0; q < g.dvt; ++q) {
    const int c0 = (quarter * g.dvt + q) * 16;
    float2 f[8];
    read16(mine + c0, f);
    store_quads(E, C, row, c0, f);
  }
  steps.wait();
  // W as tiles [dkt][parts] in the place of its right operand, and from there to the walk's copy
#pragma unroll 1
  for (int q = 0; q < g.dkt; ++q) {
    const int c0 = (quarter * g.dkt + q) * 16;
    float2 f[8];
    read16(mine + 128 + c0, f);
    put16<kP>(smem + kPrepRight + (c0 >> 6) * kP * kTile, kTile, row, c0 & 63, f);
  }
  to_async();
  before_sync();
  __syncthreads();
  if (tid == 0) {
    bulk_store(g.wimg + p.at * g.dkt * kP * kTile, base + kPrepRight, g.dkt * kP * kTile);
    bulk_commit();
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  finish(tmem, 256, steps.ok, g.status);
}

// ---- the states, chunk after chunk --------------------------------------------------------------------
//
// Forwards Z = S:  Y = E0 - W Z, kept as E;     Z <- e^G_C Z + K^T (beta e^(G_C-G) Y).
// Backwards Z = R: Y = X0 + e^(G_C-G) (K Z), kept as X;  Z <- e^G_C Z + Z0 - W^T (beta Y).
// A block walks the chunks of one head and kSlice of its dv columns; the state is in the registers of 8 warps,
// 16 columns of a row each.  The parts of Z (of Y) stand side by side as columns of one product, which reads the
// other operand once for each of its own parts.  W and K come as ready tiles in bulk copies through a ring of
// kStages, a half of an operand per stage: the first product sums over column tiles, the second over halves of
// the tokens.
//
// Bound by the chain of a chunk: two products, each with the way from tensor memory through registers into the next
// one's operand.
constexpr int kSlice = 32, kStages = 3, kChainThreads = 320;
constexpr uint32_t kStage = kP * kTile, kChainZ = kStages * kStage, kChainY = kChainZ + 2 * kTile,
                   kChainTab = kChainY + 2 * kTile;
struct ChainTab {
  uint64_t full[kStages], empty[kStages], z_ready, y_full, y_ready, z_full;
  uint32_t tmem;
};
static_assert(kChainTab + sizeof(ChainTab) <= 227 * 1024, "shared memory");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// PK: parts of K.
template <int PK, bool REV>
__global__ void __launch_bounds__(kChainThreads, 1) gd_chain_kernel(const __grid_constant__ Args g) {
  constexpr int P1 = REV ? PK : kP, P2 = REV ? kP : PK;  // parts of the two left operands
  extern __shared__ __align__(1024) unsigned char smem[];
  ChainTab& tab = *reinterpret_cast<ChainTab*>(smem + kChainTab);
  const GdArgs& a = g.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int local = blockIdx.x, bh = g.bh0 + local, b = bh / a.H, col0 = blockIdx.y * kSlice;
  const int len = length_of(a, b), chunks = (len + C - 1) / C;
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {
    if (tid == 0) atomicExch(g.status, 1);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&tab.full[i], 1);
      mbar_init(&tab.empty[i], 1);
    }
    mbar_init(&tab.z_ready, 8);
    mbar_init(&tab.y_full, 1);
    mbar_init(&tab.y_ready, 8);
    mbar_init(&tab.z_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tab.tmem)), "r"(256)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tmem = tab.tmem;
  bool ok = true;
  auto chunk_of = [&](int i) { return REV ? chunks - 1 - i : i; };
  auto tokens_of = [&](int c) { return min(C, len - c * C); };
  auto at_of = [&](int c) { return (size_t)local * g.chunks + c; };

  if (warp == 8) {
    if (elected()) {
      int turn = 0;
      auto stage = [&](uint32_t bytes) {
        const int s = turn % kStages;
        if (turn >= kStages) seq_wait(&tab.empty[s], (turn / kStages - 1) & 1, ok);
        mbar_arrive_expect_tx(&tab.full[s], bytes);
        ++turn;
        return s;
      };
      for (int i = 0; i < chunks; ++i) {
        const int c = chunk_of(i);
        const unsigned char* w = g.wimg + at_of(c) * g.dkt * kP * kTile;
        const unsigned char* k = g.kimg + at_of(c) * g.dkt * PK * kTile;
        const unsigned char *first = REV ? k : w, *second = REV ? w : k;
        for (int ct = 0; ct < g.dkt; ++ct) {
          const int s = stage(P1 * kTile);
          bulk_load(base + s * kStage, first + ct * P1 * kTile, P1 * kTile, &tab.full[s]);
        }
        for (int hf = 0; hf * 64 < tokens_of(c); ++hf) {
          const int s = stage(P2 * g.dkt * kTile / 2);
          for (int p = 0; p < P2; ++p)
            for (int ct = 0; ct < g.dkt; ++ct)
              bulk_load(base + s * kStage + (p * g.dkt + ct) * (kTile / 2),
                        second + (ct * P2 + p) * kTile + hf * (kTile / 2), kTile / 2, &tab.full[s]);
        }
      }
      for (int i = max(0, turn - kStages); i < turn; ++i) {  // every load lands before the block leaves
        bool landed = true;
        seq_wait(&tab.full[i % kStages], (i / kStages) & 1, landed);
        ok = ok && landed;
      }
    }
  } else if (warp == 9) {
    if (elected()) {
      int turn = 0;
      // D = left (PL parts) times the parts of the right side by side: the first part of the left meets all three
      auto multiply = [&](auto parts, uint32_t d, const Operand& left, const Operand& right, int k_right, int steps,
                          uint32_t id, bool add) {
        constexpr int PL = decltype(parts)::value;
#pragma unroll
        for (int p = 0; p < PL; ++p)
          for (int k = 0; k < steps; ++k)
            umma_f16(d, left.at(p, k), right.at(0, k_right + k), bf16_idesc(128, (kP - p) * kSlice) | id,
                     add || p > 0 || k > 0);
      };
      const Operand Z = mn_major(base + kChainZ, 0, kTile), Y = mn_major(base + kChainY, 0, kTile);
      for (int i = 0; i < chunks; ++i) {
        const int c = chunk_of(i);
        seq_wait(&tab.z_ready, i & 1, ok);
        after_sync();
        for (int ct = 0; ct < g.dkt; ++ct, ++turn) {
          const int s = turn % kStages;
          seq_wait(&tab.full[s], (turn / kStages) & 1, ok);
          multiply(std::integral_constant<int, P1>(), tmem, k_major(base + s * kStage, kTile, kTile), Z, 4 * ct,
                   min(4, (a.dk - 64 * ct + 15) / 16), kBMn, ct > 0);
          umma_commit(&tab.empty[s]);
        }
        umma_commit(&tab.y_full);
        seq_wait(&tab.y_ready, i & 1, ok);
        after_sync();
        for (int hf = 0; hf * 64 < tokens_of(c); ++hf, ++turn) {
          const int s = turn % kStages;
          seq_wait(&tab.full[s], (turn / kStages) & 1, ok);
          multiply(std::integral_constant<int, P2>(), tmem + 128,
                   mn_major(base + s * kStage, g.dkt * (kTile / 2), kTile / 2), Y, 4 * hf, 4, kAMn | kBMn, hf > 0);
          umma_commit(&tab.empty[s]);
        }
        umma_commit(&tab.z_full);
      }
      // every product has read its operands before the block leaves: the workers wait for the last
    }
  } else {
    const int row = (warp & 3) * 32 + lane, half = warp >> 2, c0 = col0 + half * 16;
    const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 16;
    const int rows = 64 * g.dkt, cols = 64 * g.dvt;
    const size_t head = (size_t)bh * a.dk * a.dv;
    float2 Z[8];
    const float* from = REV ? a.d_state_out : a.state;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float z[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        z[j] = from && row < a.dk && c0 + 2 * i + j < a.dv ? from[head + (size_t)row * a.dv + c0 + 2 * i + j] : 0.f;
      Z[i] = make_float2(z[0], z[1]);
    }
    auto keep = [&](float* states, size_t slot) {
      if (row < rows) store_quads(states + slot * rows * cols, rows, row, c0, Z);
    };
    auto publish = [&](uint32_t where, const float2 (&v)[8]) {  // columns [32 p, 32 p + 32) are part p's
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 w[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          uint4 u;
          u.x = take<bf16>(w[0]);
          u.y = take<bf16>(w[1]);
          u.z = take<bf16>(w[2]);
          u.w = take<bf16>(w[3]);
          const int chunk = (p & 1) * 4 + half * 2 + j;
          *reinterpret_cast<uint4*>(smem + where + (p >> 1) * kTile + row * 128 + ((chunk ^ (row & 7)) << 4)) = u;
        }
      }
      to_async();
      before_sync();
    };
    auto sum = [&](uint32_t at, float2 (&v)[8]) {
      float2 x[8], y[8];
      read16(at + 2 * kSlice, x);
      read16(at + kSlice, y);
      read16(at, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = add2(v[i], add2(y[i], x[i]));
    };
    auto fetch = [&](const float* m, int R, float2 (&v)[8]) {
      const float4* q = reinterpret_cast<const float4*>(m) + ((size_t)(c0 / 4) * R + row);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = q[(size_t)i * R];
        v[2 * i] = make_float2(f.x, f.y);
        v[2 * i + 1] = make_float2(f.z, f.w);
      }
    };
    for (int i = 0; i < chunks; ++i) {
      const int c = chunk_of(i);
      publish(kChainZ, Z);
      warp_arrive(&tab.z_ready);
      if (REV) keep(g.R, at_of(c));
      else keep(g.S, (size_t)local * (g.chunks + 1) + c);
      const Gates& gate = g.gates[at_of(c)];
      const float down = gate.down[row], beta = gate.beta[row], whole = gate.up[C - 1];
      float* ym = (REV ? g.X : g.E) + at_of(c) * C * cols;
      float2 y[8], v[8], z0[8];
      fetch(ym, C, y);
      if (REV && row < rows) fetch(g.Z0 + at_of(c) * rows * cols, rows, z0);
      seq_wait(&tab.y_full, i & 1, ok);
      __syncwarp();
      after_sync();
      sum(mine, v);
      const float2 f = both(REV ? down : -1.f), w = both(REV ? -beta : beta * down);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = fma2(f, v[j], y[j]);
        v[j] = mul2(w, y[j]);
      }
      publish(kChainY, v);
      warp_arrive(&tab.y_ready);
      store_quads(ym, C, row, c0, y);
      seq_wait(&tab.z_full, i & 1, ok);
      __syncwarp();
      after_sync();
      sum(mine + 128, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (REV) v[j] = add2(v[j], z0[j]);
        Z[j] = fma2(both(whole), Z[j], v[j]);
      }
    }
    if (!REV) keep(g.S, (size_t)local * (g.chunks + 1) + chunks);
    float* to = REV ? a.d_state : a.state_out;
    if (to && row < a.dk)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c0 + i < a.dv) to[head + (size_t)row * a.dv + c0 + i] = i & 1 ? Z[i / 2].y : Z[i / 2].x;
  }
  if (!ok) atomicExch(g.status, 1);
  before_sync();
  __syncthreads();
  if (warp == 9) {
    after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
  }
}

// ---- outputs: o = scale (e^G Q S0 + ((Q K^T) o D) U), for a chunk of a head per block -----------------------
template <typename T>
struct OutCfg {
  static constexpr int DP = kData<T>, PC = DP == 3 ? 3 : 2;
  static constexpr uint32_t kK = DP * kTile, kS = 2 * DP * kTile, kU = PC * 2 * kTile;
  static constexpr uint32_t kFirst = kS + PC * kTile, kSecond = kU + PC * kTile;
  static constexpr uint32_t kTab = kFirst > kSecond ? kFirst : kSecond;
};
struct OutTab {
  Gates gates;
  uint64_t bar;
  uint32_t tmem;
};

constexpr int kOutThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kOutThreads, kData<T> == 3 ? 1 : 2)
    gd_outputs_kernel(const __grid_constant__ Args g, bool out_vec) {
  using K = OutCfg<T>;
  constexpr int DP = K::DP, PC = K::PC, NT = kOutThreads;
  extern __shared__ __align__(1024) unsigned char smem[];
  OutTab& tab = *reinterpret_cast<OutTab*>(smem + K::kTab);
  const GdArgs& a = g.a;
  const Place p = place_of(g);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = (warp & 3) * 32 + lane, half = warp >> 2;
  T* o = static_cast<T*>(a.o) + p.b * a.ob + p.h * a.oh;
  const int live = (int)(a.T - p.t0 < C ? a.T - p.t0 : C);  // rows of the tensor
  for (int i = tid; i < (live - p.n) * a.dv; i += NT)       // zeros past the length
    o[(p.t0 + p.n + i / a.dv) * a.ot + i % a.dv] = from_f32<T>(0.f);
  if (p.n == 0) return;
  const int rows = 64 * g.dkt, cols = 64 * g.dvt;
  const float* S = g.S + p.slot * rows * cols;
  const T *q = rows_of<T>(a.q, p.t0, p.b, p.hq), *k = rows_of<T>(a.k, p.t0, p.b, p.hq);
  DataRows<T, C, 1, NT> qs, ks;
  QuadRows<64, 2, NT> ss;
  auto fetch = [&](int ct) {
    qs.fetch(q, a.q.st, 0, p.n, ct * 64, a.dk, 1, g.vec);
    ks.fetch(k, a.k.st, 0, p.n, ct * 64, a.dk, 1, g.vec);
    ss.fetch(S + ct * 64 * 4, rows, 64, g.dvt);
  };
  fetch(0);
  if (!begin(&tab.bar, &tab.tmem, 256, smem, g.status)) return;
  Steps steps{&tab.bar};
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16), base = smem_u32(smem);
  copy_gates<NT>(tab.gates, g.gates + p.at);
  for (int ct = 0; ct < g.dkt; ++ct) {
    qs.template place<DP>(smem, kTile, kTile);
    ks.template place<DP>(smem + K::kK, kTile, kTile);
    // 64 rows of the state: tiles [parts][dvt][64][64]
    ss.template place<PC>(smem + K::kS, g.dvt * (kTile / 2), kTile / 2, 64, g.dvt);
    steps.run([&] {
      const Operand Q = k_major(base, kTile, kTile);
      const int n = min(4, (a.dk - 64 * ct + 15) / 16);
      product<DP, DP>(tmem, Q, k_major(base + K::kK, kTile, kTile), n, id_of(128, false, false), ct > 0);
      product<DP, PC>(tmem + 128, Q, mn_major(base + K::kS, g.dvt * (kTile / 2), kTile / 2), n,
                      id_of(cols, false, true), ct > 0);
    });
    if (ct + 1 < g.dkt) fetch(ct + 1);
    steps.wait();
  }
  QuadRows<C, 1, NT> es;
  const float* E = g.E + p.at * C * cols;
  es.fetch(E, C, C, 1);
  {
    const float hi = tab.gates.hi[row], lo = tab.gates.lo[row];
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
      const int c0 = half * 64 + x * 16;
      float2 v[8];
      read16(mine + c0, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = c0 + 2 * i;
        v[i].x = j <= row ? v[i].x * decay_between(hi, lo, tab.gates.hi[j], tab.gates.lo[j]) : 0.f;
        v[i].y = j < row ? v[i].y * decay_between(hi, lo, tab.gates.hi[j + 1], tab.gates.lo[j + 1]) : 0.f;
      }
      put16<PC>(smem, 2 * kTile, row, c0, v);
    }
  }
  const float up = tab.gates.up[row];
  for (int vt = 0; vt < g.dvt; ++vt) {
    es.template place<PC>(smem + K::kU, kTile, kTile, C, 1, tab.gates.beta);
    steps.run([&] {
      product<PC, PC>(tmem, k_major(base, 2 * kTile, kTile), mn_major(base + K::kU, kTile, kTile), 8,
                      id_of(64, false, true), false);
    });
    if (vt + 1 < g.dvt) es.fetch(E + (size_t)(vt + 1) * 16 * C * 4, C, C, 1);
    steps.wait();
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      const int c = half * 32 + x * 16, c0 = vt * 64 + c;
      float2 v[8], w[8];
      read16(mine + c, v);
      read16(mine + 128 + c0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mul2(fma2(both(up), w[i], v[i]), both(a.scale));
      if (row < p.n) store16<T>(o + (p.t0 + row) * a.ot + c0, a.dv - c0, out_vec, v);
    }
  }
  finish(tmem, 256, steps.ok, g.status);
}

template <typename K>
cudaError_t allow(K kernel, uint32_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

}  // namespace

cudaError_t launch_prepare(const Args& g, bool keep_inverse, cudaStream_t s) {
  PRNN_BY_DTYPE(g.a.dtype, T, {
    constexpr uint32_t smem = kPrepTab + sizeof(PrepTab);
    const cudaError_t e = allow(gd_prepare_kernel<T>, smem);
    if (e != cudaSuccess) return e;
    gd_prepare_kernel<T><<<(unsigned)(g.nbh * g.chunks), kPrepThreads, smem, s>>>(g, keep_inverse);
  });
  return cudaGetLastError();
}

cudaError_t launch_chain(const Args& g, bool reverse, cudaStream_t s) {
  constexpr uint32_t smem = kChainTab + sizeof(ChainTab);
  const dim3 grid(g.nbh, (g.a.dv + kSlice - 1) / kSlice);
  PRNN_BY_DTYPE(g.a.dtype, T, {
    constexpr int PK = kData<T>;
    const cudaError_t e = reverse ? allow(gd_chain_kernel<PK, true>, smem) : allow(gd_chain_kernel<PK, false>, smem);
    if (e != cudaSuccess) return e;
    if (reverse) gd_chain_kernel<PK, true><<<grid, kChainThreads, smem, s>>>(g);
    else gd_chain_kernel<PK, false><<<grid, kChainThreads, smem, s>>>(g);
  });
  return cudaGetLastError();
}

cudaError_t launch_outputs(const Args& g, cudaStream_t s) {
  PRNN_BY_DTYPE(g.a.dtype, T, {
    constexpr uint32_t smem = OutCfg<T>::kTab + sizeof(OutTab);
    const cudaError_t e = allow(gd_outputs_kernel<T>, smem);
    if (e != cudaSuccess) return e;
    constexpr int V = 16 / sizeof(T);
    const bool vec = (reinterpret_cast<uintptr_t>(g.a.o) & 15) == 0 && (g.a.T == 1 || g.a.ot % V == 0) &&
                     (g.a.B == 1 || g.a.ob % V == 0) && (g.a.H == 1 || g.a.oh % V == 0);
    gd_outputs_kernel<T><<<(unsigned)(g.nbh * g.chunks), kOutThreads, smem, s>>>(g, vec);
  });
  return cudaGetLastError();
}

}  // namespace gd

namespace {

using namespace gd;

size_t up16(size_t n) { return (n + 15) / 16 * 16; }
struct Plan {
  int chunks, dkt, dvt, nbh;
  size_t w, k, gates, E, S, inv, X, Z0, R, total;  // bytes of each part for nbh heads
};
// Heads go together in groups whose scratch stays within kMost bytes (one head at least).
constexpr size_t kMost = (size_t)8 << 30;
Plan plan_of(prnn_dtype_t dtype, int T, int B, int H, int dk, int dv, bool backward) {
  Plan p{};
  p.chunks = (T + C - 1) / C;
  p.dkt = (dk + 63) / 64;
  p.dvt = (dv + 63) / 64;
  const size_t n = p.chunks, parts = dtype == PRNN_F32 ? 3 : (dtype == PRNN_F16 ? 2 : 1);
  const size_t rows = 64 * p.dkt, cols = 64 * p.dvt;
  const size_t w = n * p.dkt * kP * kTile, k = n * p.dkt * parts * kTile, gates = n * sizeof(Gates), E = n * C * cols * 4,
               S = (n + 1) * rows * cols * 4, inv = n * C * C * 4, Z0 = n * rows * cols * 4;
  const size_t one = w + k + gates + E + S + (backward ? inv + E + 2 * Z0 : 0);
  p.nbh = (int)std::min<size_t>((size_t)B * H, std::max<size_t>(1, kMost / one));
  // the heads of a group times their chunks are one grid
  p.nbh = (int)std::min<size_t>(p.nbh, 0x7fffffff / n);
  const size_t m = p.nbh;
  p.w = m * w;
  p.k = m * k;
  p.gates = up16(m * gates);
  p.E = m * E;
  p.S = m * S;
  p.inv = backward ? m * inv : 0;
  p.X = backward ? m * E : 0;
  p.Z0 = p.R = backward ? m * Z0 : 0;
  p.total = p.w + p.k + p.gates + p.E + p.S + p.inv + p.X + p.Z0 + p.R;
  return p;
}

bool seq_vec(const LaSeq& s, const GdArgs& a, int d, int heads) {
  const int v = a.dtype == PRNN_F32 ? 4 : 8;
  return (reinterpret_cast<uintptr_t>(s.p) & 15) == 0 && d % 8 == 0 && (a.T == 1 || s.st % v == 0) &&
         (a.B == 1 || s.sb % v == 0) && (heads == 1 || s.sh % v == 0);
}

}  // namespace

bool gd_tc_serves(prnn_dtype_t, int T, int dk, int dv) { return dk <= 128 && dv <= 128 && T >= kGdTcLeast; }

size_t gd_tc_workspace(prnn_dtype_t dtype, int T, int B, int H, int dk, int dv, bool backward) {
  return plan_of(dtype, T, B, H, dk, dv, backward).total;
}

cudaError_t launch_gd_tc(const GdArgs& a, void* scratch, bool backward, cudaStream_t s) {
  const Plan p = plan_of(a.dtype, a.T, a.B, a.H, a.dk, a.dv, backward);
  Args g{};
  g.a = a;
  g.chunks = p.chunks;
  g.dkt = p.dkt;
  g.dvt = p.dvt;
  g.status = seq_status_word();
  if (!g.status) return cudaErrorUnknown;
  const int hq = a.H / a.q.share;
  g.vec = seq_vec(a.q, a, a.dk, hq) && seq_vec(a.k, a, a.dk, hq) && seq_vec(a.v, a, a.dv, a.H) &&
          (!backward || seq_vec(a.d_o, a, a.dv, a.H));
  char* at = static_cast<char*>(scratch);
  auto take = [&](size_t n) {
    char* here = at;
    at += n;
    return reinterpret_cast<float*>(here);
  };
  g.wimg = reinterpret_cast<unsigned char*>(take(p.w));
  g.kimg = reinterpret_cast<unsigned char*>(take(p.k));
  g.gates = reinterpret_cast<Gates*>(take(p.gates));
  g.E = take(p.E);
  g.S = take(p.S);
  g.inv = take(p.inv);
  g.X = take(p.X);
  g.Z0 = take(p.Z0);
  g.R = take(p.R);
  for (g.bh0 = 0; g.bh0 < a.B * a.H; g.bh0 += p.nbh) {
    g.nbh = std::min(p.nbh, a.B * a.H - g.bh0);
    cudaError_t e = launch_prepare(g, backward, s);
    if (e == cudaSuccess) e = launch_chain(g, false, s);
    if (e == cudaSuccess && !backward) e = launch_outputs(g, s);
    if (e == cudaSuccess && backward) e = launch_before_reverse(g, s);
    if (e == cudaSuccess && backward) e = launch_chain(g, true, s);
    if (e == cudaSuccess && backward) e = launch_gradients(g, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace prnn
