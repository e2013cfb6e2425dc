// gated_delta_tc.cu -- the gated delta rule's forward pass in chunks on the 5th-generation tensor cores, and the plan of
// its backward pass.  The algebra and the rounding are in gated_delta_tc.cuh.
#include <algorithm>

#include "gated_delta_tc.cuh"

namespace prnn {
namespace gd {
namespace {

// ---- before the states: gates, Tt, Tt V, W, for a chunk of a head at a time --------------------------------
//
// Tt is the inverse of I + A, A strictly lower triangular.  The diagonal blocks of 32 go by substitution, a column per
// lane; those of 64 from them by T_10 = -T_11 A_10 T_00 in fp32; and the last block of 64 by the same formula
// on the tensor cores.
//
// The steps stand one behind another, so two blocks share an SM and fill each other's waits.  That fits because Tt is kept
// without its zero quarter: its columns 64 ... have rows 64 ... only, as the left operand of a sum of their own that
// counts in those rows alone (the 64 rows before them, which the product reads as well, hold anything); and
// because right operands come in pieces of 64 tokens.  Where chunks are too few for that, one block of twice the threads and
// with whole right operands takes a chunk in less time: 180 chunks of fp32, of which a half are empty, 27 us against 41;
// but 2048 of bf16 264 us against 235.
constexpr int kLd = 68;  // floats of a row of 64: 16-byte aligned, rows a quad of banks apart
struct PrepTab {
  Gates gates;
  double part[4];
  uint64_t bar;
  uint32_t tmem;
};
// Tt's columns 0 ... and 64 ... as parts, a right operand.  Before them, in the same place: K; A and T in fp32 with A_10 as
// parts.  After them: W.
constexpr uint32_t kHalf = kTile / 2, kTt1 = kP * kTile, kPrepT = 2 * 64 * kLd * 4, kPrepRight = kTt1 + kP * kHalf;
template <int NT>
constexpr uint32_t kPrepTab = kPrepRight + (NT == 512 ? 2 * kP * kTile : kP * kHalf);
static_assert(2 * kPrepT <= kPrepRight && 2 * kP * kTile <= kPrepTab<256> &&
                  2 * (kPrepTab<256> + sizeof(PrepTab) + 1024) <= 228 * 1024 &&
                  kPrepTab<512> + sizeof(PrepTab) <= 227 * 1024,
              "shared memory of two blocks, and of one");

// T_10 <- -T_11 (A_10 T_00) of 2 x 2 blocks of 32, for two diagonal blocks of 64; the product in brackets is kept in
// T's unused block (0, 1).
template <int NT>
__device__ __forceinline__ void lower_blocks(const float* A, float* T) {
  constexpr int Q = NT / 2, X = 512 / Q;  // threads of a block of 64, rows of 2 values each
  const int q = threadIdx.x % Q, r = (q >> 4) * X, c = (q & 15) * 2;
  A += threadIdx.x / Q * 64 * kLd;
  T += threadIdx.x / Q * 64 * kLd;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const float* left = pass == 0 ? A + (32 + r) * kLd : T + (32 + r) * kLd + 32;
    const float* right = pass == 0 ? T + c : T + 32 + c;
    float2 s[X];
#pragma unroll
    for (int x = 0; x < X; ++x) s[x] = both(0.f);
#pragma unroll 4
    for (int m = 0; m < 32; m += 4) {
      float2 f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = *reinterpret_cast<const float2*>(right + (m + k) * kLd);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const float4 l = *reinterpret_cast<const float4*>(left + x * kLd + m);
        s[x] = fma2(both(l.w), f[3], fma2(both(l.z), f[2], fma2(both(l.y), f[1], fma2(both(l.x), f[0], s[x]))));
      }
    }
    float* to = pass == 0 ? T + r * kLd + 32 + c : T + (32 + r) * kLd + c;
#pragma unroll
    for (int x = 0; x < X; ++x)
      *reinterpret_cast<float2*>(to + x * kLd) = pass == 0 ? s[x] : mul2(s[x], both(-1.f));
    __syncthreads();
  }
}

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's own stores have read their source.
__device__ __forceinline__ void bulk_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) gd_prepare_kernel(const __grid_constant__ Args g, int keep_inverse) {
  constexpr int DP = kData<T>, VT = DP == 1 ? 2 : 1;  // tiles of V in a piece
  constexpr int GROUPS = NT / C, BLOCKS = 4 / GROUPS;  // groups of columns, blocks of 16 of 64 columns for each
  constexpr bool kWhole = NT == 512;
  extern __shared__ __align__(1024) unsigned char smem[];
  PrepTab& tab = *reinterpret_cast<PrepTab*>(smem + kPrepTab<NT>);
  const GdArgs& a = g.a;
  int index = blockIdx.x;
  Place p = next_place(g, index);
  if (p.n == 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = (warp & 3) * 32 + lane, group = warp >> 2;
  const bool low = (warp & 3) >= 2;  // rows 64 ...
  auto keys = [&](const Place& at) { return rows_of<T>(a.k, at.t0, at.b, at.hq); };
  DataRows<T, C, 2, NT> rows;
  rows.fetch(keys(p), a.k.st, 0, p.n, 0, a.dk, g.dkt);
  if (!begin(&tab.bar, &tab.tmem, 256, smem, g.status)) return;
  Steps steps{&tab.bar};
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16), base = smem_u32(smem);
  const uint32_t part = g.dkt * kTile;
  // Tt's columns 0 ... and, with rows 0 ... 63 that do not count, 64 ...
  const Operand left0 = k_major(base, kTile, kTile), left1 = k_major(base + kTt1 - kHalf, kHalf, kTile);
  float *A = reinterpret_cast<float*>(smem), *inv = reinterpret_cast<float*>(smem + kPrepT);
  float gate = 0.f, beta = 0.f;
  auto ask_gates = [&](const Place& at) {
    const long long t = at.t0 + tid;
    const bool in = tid < at.n;
    gate = in ? a.g[t * a.gt + at.b * a.gb + at.h * a.gh] : 0.f;
    beta = in ? a.beta[t * a.bt + at.b * a.bb + at.h * a.bh] : 0.f;
  };
  // columns c0 ... of an accumulator whose tokens 64 ... have one of their own, 128 columns on
  auto read_both = [&](int c0, int n, float2 (&v)[8]) {
    read16(mine + c0, v);
    if (low && n > 64) {
      float2 x[8];
      read16(mine + 128 + c0, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = add2(v[i], x[i]);
    }
  };
  ask_gates(p);
  while (p.n > 0) {
    const Place at = p;
    double G = 0;
    if (tid < C) {
      if (gate < -1000.f) gate = -1000.f;
      G = gate * 1.4426950408889634;
      tab.gates.beta[tid] = beta;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, G, o);
        if (lane >= o) G += x;
      }
      if (lane == 31) tab.part[warp] = G;
    }
    if (tid == 0) bulk_read();  // the last chunk's W
    __syncthreads();
    rows.template place<DP>(smem, part, kTile);
    if (tid < C) {
      double all = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w < warp) G += tab.part[w];
        all += tab.part[w];
      }
      const double last = __shfl_sync(0xffffffffu, G, lane | 15);
      const float hi = (float)G;
      tab.gates.sum[tid] = make_float2(hi, (float)(G - hi));
      tab.gates.up[tid] = exp2f(hi);
      tab.gates.down[tid] = exp2f((float)(all - G));
      tab.gates.to_last[tid] = exp2f((float)(last - G));
    }
    const Operand K = k_major(base, part, kTile);
    steps.run([&] { product<DP, DP>(tmem, K, K, (a.dk + 15) / 16, id_of(128, false, false), false); });
    if (tid == 0) {  // the walk's copy of K
      for (int ct = 0; ct < g.dkt; ++ct)
        for (int q = 0; q < DP; ++q)
          bulk_store(g.kimg + ((at.at * g.dkt + ct) * DP + q) * kTile, base + q * part + ct * kTile, kTile);
      bulk_commit();
    }
    {
      const float* from = reinterpret_cast<const float*>(&tab.gates);
      float* to = reinterpret_cast<float*>(g.gates + at.at);
      for (int i = tid; i < (int)(sizeof(Gates) / 4); i += NT) to[i] = from[i];
    }
    if (tid == 0) bulk_read();
    steps.wait();
    __syncthreads();  // K's place may be written
#pragma unroll 1
    for (int q = 0; q < 2 * BLOCKS; ++q) {  // A_ij = (k_i . k_j) D_ij beta_j below the diagonal
      const int c0 = (group * 2 * BLOCKS + q) * 16;
      if ((c0 >> 5) > (warp & 3)) continue;  // behind all of the warp's rows
      float2 x[8];
      read16(mine + c0, x);
      decayed<true>(x, row, c0, tab.gates);
      times16(x, tab.gates.beta + c0);
      if (low && c0 < 64) {
        put16<kP>(smem + kPrepRight, kHalf, row - 64, c0, x);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(A + row * kLd + (c0 & 63) + 4 * i) =
              make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
      }
    }
    before_sync();
    __syncthreads();
    if (warp < 4) {
      float x[32];
      const int r0 = 32 * warp, c0 = 32 * (warp & 1);
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        float s[4] = {r == lane ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < r; m += 4) {
          const float4 l = *reinterpret_cast<const float4*>(A + (r0 + r) * kLd + c0 + m);
          s[0] = fmaf(-l.x, x[m], s[0]);
          if (m + 1 < r) s[1] = fmaf(-l.y, x[m + 1], s[1]);
          if (m + 2 < r) s[2] = fmaf(-l.z, x[m + 2], s[2]);
          if (m + 3 < r) s[3] = fmaf(-l.w, x[m + 3], s[3]);
        }
        x[r] = (s[0] + s[1]) + (s[2] + s[3]);
        inv[(r0 + r) * kLd + c0 + lane] = x[r];
      }
    }
    __syncthreads();
    lower_blocks<NT>(A, inv);
    {  // the diagonal blocks of 64 as parts, in the place of themselves and A
      float2 x[BLOCKS][8];
      const int col0 = (low ? 64 : 0) + group * BLOCKS * 16;
#pragma unroll
      for (int q = 0; q < BLOCKS; ++q)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const int c = col0 + q * 16 + 2 * i;
          const float4 f = *reinterpret_cast<const float4*>(inv + row * kLd + (c & 63));
          x[q][i] = make_float2(c <= row ? f.x : 0.f, c + 1 <= row ? f.y : 0.f);
          x[q][i + 1] = make_float2(c + 2 <= row ? f.z : 0.f, c + 3 <= row ? f.w : 0.f);
        }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < BLOCKS; ++q) {
        const int c0 = col0 + q * 16;
        if (low) put16<kP>(smem + kTt1, kHalf, row - 64, c0 - 64, x[q]);
        else put16<kP>(smem, kTile, row, c0, x[q]);
        if (!keep_inverse) continue;
        store_quads(g.inv + at.at * C * C, C, row, c0, x[q]);
        if (low) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[q][i] = both(0.f);
        store_quads(g.inv + at.at * C * C, C, row, c0 + 64, x[q]);
      }
    }
    // T_10: A_10 T_00, whose rows 64 ... count, then T_11 times that
    steps.run([&] {
      product<kP, kP>(tmem + 128, k_major(base + kPrepRight - kHalf, kHalf, kTile), mn_major(base, kTile, kTile), 4,
                      id_of(64, false, true), false);
    });
    steps.wait();
    if (low)
#pragma unroll 1
      for (int q = 0; q < BLOCKS; ++q) {
        const int c0 = (group * BLOCKS + q) * 16;
        float2 x[8];
        read16(mine + 128 + c0, x);
        put16<kP>(smem + kPrepRight, kHalf, row - 64, c0, x);
      }
    const Operand right = mn_major(base + kPrepRight, kHalf, kHalf);
    steps.run([&] { product<kP, kP>(tmem + 192, left1, right, 4, id_of(64, false, true), false); });
    DataRows<T, 64, VT, NT> vs;
    const T* v = rows_of<T>(a.v, at.t0, at.b, at.h);
    if constexpr (kWhole) rows.fetch(v, a.v.st, 0, at.n, 0, a.dv, g.dvt);
    else vs.fetch(v, a.v.st, 0, at.n, 0, a.dv, VT == 2 ? g.dvt : 1);
    steps.wait();
    if (low)
#pragma unroll 1
      for (int q = 0; q < BLOCKS; ++q) {
        const int c0 = (group * BLOCKS + q) * 16;
        float2 x[8];
        read16(mine + 192 + c0, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], both(-1.f));
        put16<kP>(smem, kTile, row, c0, x);
        if (keep_inverse) store_quads(g.inv + at.at * C * C, C, row, c0, x);
      }
    // Tt V, tokens 64 ... in columns 128 ...
    const int vpieces = VT == 2 ? 1 : g.dvt;
    DataRows<T, 64, 1, NT> ks;
    // a whole right operand of `tiles` tiles, its tokens 64 ... for columns 128 ...
    auto whole = [&](auto parts, int tiles) {
      constexpr int PR = decltype(parts)::value;
      steps.run([&] {
        Operand both_halves = mn_major(base + kPrepRight, tiles * kTile, kTile);
        product<kP, PR>(tmem, left0, both_halves, 4, id_of(64 * tiles, false, true), false);
        both_halves.desc += kHalf >> 4;
        if (at.n > 64) product<kP, PR>(tmem + 128, left1, both_halves, 4, id_of(64 * tiles, false, true), false);
      });
    };
    if constexpr (kWhole) {
      rows.template place<DP>(smem + kPrepRight, g.dvt * kTile, kTile);
      whole(std::integral_constant<int, DP>(), g.dvt);
      rows.fetch(keys(at), a.k.st, 0, at.n, 0, a.dk, g.dkt);
      steps.wait();
    }
#pragma unroll 1
    for (int i = 0; !kWhole && i < 2 * vpieces && i / vpieces * 64 < at.n; ++i) {
      const int th = i / vpieces, vt = i % vpieces;
      vs.template place<DP>(smem + kPrepRight, VT == 2 ? 0 : kHalf, kHalf);
      steps.run([&] {
        product<kP, DP>(tmem + 128 * th + 64 * vt, th ? left1 : left0, right, 4,
                        id_of(VT == 2 ? 64 * g.dvt : 64, false, true), false);
      });
      const int next = i + 1, nh = next / vpieces;
      if (nh < 2 && nh * 64 < at.n) vs.fetch(v, a.v.st, nh * 64, at.n, next % vpieces * 64, a.dv, VT == 2 ? g.dvt : 1);
      else ks.fetch(keys(at), a.k.st, 0, at.n, 0, a.dk, 1);
      steps.wait();
    }
    float* E = g.E + at.at * C * 64 * g.dvt;
#pragma unroll 1
    for (int q = 0; q < BLOCKS * g.dvt; ++q) {
      const int c0 = (group * BLOCKS * g.dvt + q) * 16;
      float2 f[8];
      read_both(c0, at.n, f);
      store_quads(E, C, row, c0, f);
    }
    // W = Tt (e^G K), likewise
    index += gridDim.x;
    p = next_place(g, index);
    if constexpr (kWhole) {
      rows.template place<kP>(smem + kPrepRight, part, kTile, tab.gates.up);
      whole(std::integral_constant<int, kP>(), g.dkt);
      if (p.n > 0) {
        rows.fetch(keys(p), a.k.st, 0, p.n, 0, a.dk, g.dkt);
        ask_gates(p);
      }
      steps.wait();
    }
#pragma unroll 1
    for (int i = 0; !kWhole && i < 2 * g.dkt && i / g.dkt * 64 < at.n; ++i) {
      const int th = i / g.dkt, ct = i % g.dkt;
      ks.template place<kP>(smem + kPrepRight, kHalf, kHalf, tab.gates.up + 64 * th);
      steps.run([&] {
        product<kP, kP>(tmem + 128 * th + 64 * ct, th ? left1 : left0, right, 4, id_of(64, false, true), false);
      });
      const int next = i + 1, nh = next / g.dkt;
      if (nh < 2 && nh * 64 < at.n) {
        ks.fetch(keys(at), a.k.st, nh * 64, at.n, next % g.dkt * 64, a.dk, 1);
      } else if (p.n > 0) {
        rows.fetch(keys(p), a.k.st, 0, p.n, 0, a.dk, g.dkt);
        ask_gates(p);
      }
      steps.wait();
    }
    // as tiles [dkt][parts], and from there to the walk's copy
#pragma unroll 1
    for (int q = 0; q < BLOCKS * g.dkt; ++q) {
      const int c0 = (group * BLOCKS * g.dkt + q) * 16;
      float2 f[8];
      read_both(c0, at.n, f);
      put16<kP>(smem + (c0 >> 6) * kP * kTile, kTile, row, c0 & 63, f);
    }
    to_async();
    before_sync();
    __syncthreads();
    if (tid == 0) {
      bulk_store(g.wimg + at.at * g.dkt * kP * kTile, base, g.dkt * kP * kTile);
      bulk_commit();
    }
  }
  if (tid == 0) bulk_read();
  finish(tmem, 256, steps.ok, g.status);
}

// ---- the states, chunk after chunk --------------------------------------------------------------------
//
// Forwards Z = S:  Y = E0 - W Z, kept as E;     Z <- e^G_C Z + K^T (beta e^(G_C-G) Y).
// Backwards Z = R: Y = X0 + e^(G_C-G) (K Z), kept as X;  Z <- e^G_C Z + Z0 - W^T (beta Y).
// A block walks the chunks of one head and SL of its dv columns; the state is in the registers of SL / 4 warps,
// 16 columns of a row each.  The parts of Z (of Y) stand side by side as columns of one product, which reads the
// other operand once for each of its own parts.  W and K come as ready tiles in bulk copies, a half of an operand at a
// time: the first product sums over column tiles, the second over halves of the tokens.
//
// Bound by the chain of a chunk: two products, each with the way from tensor memory through registers into the next
// one's operand (4600 cycles in slices of 32: T = 8192, 2 sequences of 16 heads of 128 x 128 bf16 155 us).  Slices of 32
// columns make it shorter and spread a head over more SMs; slices of 64 take half the blocks, for when those of 32 would
// not run all at once (T = 2048, 4 sequences: forward 65 us against 91, backwards 78 against 129 before it read Z0 late).
//
// Where the halves of both operands fit side by side each has a place of its own, and the next chunk's is requested as
// soon as the product with this one's has read it; else they share a ring (fp32, and fp16 in slices of 64).  What the
// workers read, Y0 and Z0, is brought into L2 a chunk ahead.
constexpr uint32_t kStage = kP * kTile;
template <int SL, int PK, bool REV>
struct ChainCfg {
  static constexpr bool kOwn = PK <= (SL == 32 ? 2 : 1);
  static constexpr int kRing = SL == 32 ? 3 : 2, kWorkers = SL / 4, kThreads = 32 * (kWorkers + 2);
  static constexpr int P1 = REV ? PK : kP, P2 = REV ? kP : PK;           // parts of the two left operands
  static constexpr uint32_t kLoads = kOwn ? 2 * (kP + PK) * kTile : kRing * kStage;
  static constexpr uint32_t kOperand = SL == 32 ? 2 * kTile : 3 * kTile;  // parts side by side in tiles of 64 columns
  static constexpr uint32_t kZ = kLoads, kY = kZ + kOperand, kTab = kY + kOperand;
  // tensor memory, used by both products in turn: the left operand's first part times all of the right one's, and the
  // small rest, which would lose more to the rounding of each step's sum beside the large ones
  static constexpr uint32_t kSmall = kP * SL, kCols = SL == 32 ? 256 : 512;
};
struct ChainTab {
  uint64_t full[4], empty[4], z_ready, y_full, y_ready, z_full;
  uint32_t tmem;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// PK: parts of K.
template <int PK, bool REV, int SL>
__global__ void __launch_bounds__((ChainCfg<SL, PK, REV>::kThreads), 1) gd_chain_kernel(const __grid_constant__ Args g) {
  using K = ChainCfg<SL, PK, REV>;
  static_assert(K::kTab + sizeof(ChainTab) <= 227 * 1024, "shared memory");
  constexpr int kWorkers = K::kWorkers, P1 = K::P1, P2 = K::P2;
  extern __shared__ __align__(1024) unsigned char smem[];
  ChainTab& tab = *reinterpret_cast<ChainTab*>(smem + K::kTab);
  const GdArgs& a = g.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int local = blockIdx.x, bh = g.bh0 + local, b = bh / a.H, col0 = blockIdx.y * SL;
  const int len = length_of(a, b), chunks = (len + C - 1) / C;
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {
    if (tid == 0) atomicExch(g.status, 1);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&tab.full[i], 1);
      mbar_init(&tab.empty[i], 1);
    }
    mbar_init(&tab.z_ready, kWorkers);
    mbar_init(&tab.y_full, 1);
    mbar_init(&tab.y_ready, kWorkers);
    mbar_init(&tab.z_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWorkers + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tab.tmem)), "r"(K::kCols)
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

  // The place of half `half` of the first or second left operand of the i-th chunk, and how many it has held before;
  // `turn` counts the ring's.
  struct Slot {
    int s, n;
    uint32_t at;
  };
  const bool short_last = chunks > 0 && tokens_of(chunks - 1) <= 64;
  auto slot = [&](int second, int half, int i, int& turn) {
    if constexpr (K::kOwn) {
      const int s = 2 * second + half;
      // the last chunk may have no second half of tokens; backwards it comes first
      return Slot{s, i - (REV && s == 3 && short_last ? 1 : 0),
                  second ? (2 * P1 + half * P2) * kTile : half * P1 * kTile};
    } else {
      const Slot at{turn % K::kRing, turn / K::kRing, turn % K::kRing * kStage};
      ++turn;
      return at;
    }
  };

  if (warp == kWorkers) {
    if (elected()) {
      int turn = 0;
      auto request = [&](const Slot& at, uint32_t bytes) {
        if (at.n > 0) seq_wait(&tab.empty[at.s], (at.n - 1) & 1, ok);
        mbar_arrive_expect_tx(&tab.full[at.s], bytes);
      };
      const int rows = 64 * g.dkt, cols = 64 * g.dvt, wide = min(SL, cols - col0);
      auto ahead = [&](int i) {
        if (i >= chunks) return;
        const size_t at = at_of(chunk_of(i));
        ask_l2((REV ? g.X : g.E) + at * C * cols + (size_t)col0 * C, wide * C * 4);
        if (REV) ask_l2(g.Z0 + at * rows * cols + (size_t)col0 * rows, wide * rows * 4);
      };
      ahead(0);
      for (int i = 0; i < chunks; ++i) {
        const int c = chunk_of(i);
        const unsigned char* w = g.wimg + at_of(c) * g.dkt * kP * kTile;
        const unsigned char* k = g.kimg + at_of(c) * g.dkt * PK * kTile;
        const unsigned char *first = REV ? k : w, *second = REV ? w : k;
        ahead(i + 1);
        for (int ct = 0; ct < g.dkt; ++ct) {
          const Slot at = slot(0, ct, i, turn);
          request(at, P1 * kTile);
          bulk_load(base + at.at, first + ct * P1 * kTile, P1 * kTile, &tab.full[at.s]);
        }
        for (int hf = 0; hf * 64 < tokens_of(c); ++hf) {
          const Slot at = slot(1, hf, i, turn);
          request(at, P2 * g.dkt * kTile / 2);
          for (int p = 0; p < P2; ++p)
            for (int ct = 0; ct < g.dkt; ++ct)
              bulk_load(base + at.at + (p * g.dkt + ct) * (kTile / 2),
                        second + (ct * P2 + p) * kTile + hf * (kTile / 2), kTile / 2, &tab.full[at.s]);
        }
      }
      // every load lands before the block leaves
      auto land = [&](int s, int n) {
        if (n < 0) return;
        bool landed = true;
        seq_wait(&tab.full[s], n & 1, landed);
        ok = ok && landed;
      };
      if constexpr (K::kOwn) {
        land(0, chunks - 1);
        land(1, g.dkt > 1 ? chunks - 1 : -1);
        land(2, chunks - 1);
        land(3, chunks - 1 - (short_last ? 1 : 0));
      } else {
        for (int i = max(0, turn - K::kRing); i < turn; ++i) land(i % K::kRing, i / K::kRing);
      }
    }
  } else if (warp == kWorkers + 1) {
    if (elected()) {
      int turn = 0;
      // left (PL parts) times the parts of the right side by side: the first part of the left meets all three
      auto multiply = [&](auto parts, const Operand& left, const Operand& right, int k_right, int steps, uint32_t id,
                          bool add) {
        constexpr int PL = decltype(parts)::value;
#pragma unroll
        for (int p = 0; p < PL; ++p)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps)
              umma_f16(tmem + (p > 0 ? K::kSmall : 0), left.at(p, k), right.at(0, k_right + k),
                       bf16_idesc(128, (kP - p) * SL) | id, add || p > 1 || k > 0);
      };
      const Operand Z = mn_major(base + K::kZ, 0, kTile), Y = mn_major(base + K::kY, 0, kTile);
      for (int i = 0; i < chunks; ++i) {
        const int c = chunk_of(i);
        seq_wait(&tab.z_ready, i & 1, ok);
        after_sync();
        for (int ct = 0; ct < g.dkt; ++ct) {
          const Slot at = slot(0, ct, i, turn);
          seq_wait(&tab.full[at.s], at.n & 1, ok);
          multiply(std::integral_constant<int, P1>(), k_major(base + at.at, kTile, kTile), Z, 4 * ct,
                   min(4, (a.dk - 64 * ct + 15) / 16), kBMn, ct > 0);
          umma_commit(&tab.empty[at.s]);
        }
        umma_commit(&tab.y_full);
        seq_wait(&tab.y_ready, i & 1, ok);
        after_sync();
        for (int hf = 0; hf * 64 < tokens_of(c); ++hf) {
          const Slot at = slot(1, hf, i, turn);
          seq_wait(&tab.full[at.s], at.n & 1, ok);
          multiply(std::integral_constant<int, P2>(), mn_major(base + at.at, g.dkt * (kTile / 2), kTile / 2), Y, 4 * hf, 4,
                   kAMn | kBMn, hf > 0);
          umma_commit(&tab.empty[at.s]);
        }
        umma_commit(&tab.z_full);
      }
      // every product has read its operands before the block leaves: the workers wait for the last
    }
  } else {
    const int row = (warp & 3) * 32 + lane, part16 = warp >> 2, c0 = col0 + part16 * 16;
    const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + part16 * 16;
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
    auto publish = [&](uint32_t where, const float2 (&v)[8]) {  // columns [SL p, SL p + SL) are part p's
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
          const int c = p * SL + part16 * 16 + j * 8, chunk = (c & 63) >> 3;
          *reinterpret_cast<uint4*>(smem + where + (c >> 6) * kTile + row * 128 + ((chunk ^ (row & 7)) << 4)) = u;
        }
      }
      to_async();
      before_sync();
    };
    auto sum = [&](bool small, float2 (&v)[8]) {  // the small ones first
      uint32_t x[16], y[16], z[16];
      if (small) {
        tmem_ld16(mine + K::kSmall + SL, x);
        tmem_ld16(mine + K::kSmall, y);
        wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = add2(pair_at(x, i), pair_at(y, i));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = both(0.f);
      }
      tmem_ld16(mine + 2 * SL, x);
      tmem_ld16(mine + SL, y);
      tmem_ld16(mine, z);
      wait_ld();
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = add2(add2(v[i], add2(pair_at(x, i), pair_at(y, i))), pair_at(z, i));
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
      publish(K::kZ, Z);
      warp_arrive(&tab.z_ready);
      if (REV) keep(g.R, at_of(c));
      else keep(g.S, (size_t)local * (g.chunks + 1) + c);
      const Gates& gate = g.gates[at_of(c)];
      const float down = gate.down[row], beta = gate.beta[row], whole = gate.up[C - 1];
      float* ym = (REV ? g.X : g.E) + at_of(c) * C * cols;
      float2 y[8], v[8], z0[8];
      fetch(ym, C, y);
      seq_wait(&tab.y_full, i & 1, ok);
      __syncwarp();
      after_sync();
      sum(P1 > 1, v);
      const float2 f = both(REV ? down : -1.f), w = both(REV ? -beta : beta * down);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = fma2(f, v[j], y[j]);
        v[j] = mul2(w, y[j]);
      }
      publish(K::kY, v);
      warp_arrive(&tab.y_ready);
      store_quads(ym, C, row, c0, y);
      if (REV && row < rows) fetch(g.Z0 + at_of(c) * rows * cols, rows, z0);
      seq_wait(&tab.z_full, i & 1, ok);
      __syncwarp();
      after_sync();
      sum(P2 > 1, v);
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
  if (warp == kWorkers + 1) {
    after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(K::kCols) : "memory");
  }
}

// ---- outputs: o = scale (e^G Q S0 + ((Q K^T) o D) U), for a chunk of a head per block -----------------------
//
// Computed operands have two parts where the output has 16 bits (three in fp32): two blocks share an SM.  T = 8192, 2
// sequences of 16 heads of 128 x 128 bf16: 152 us, the steps' latency; all pairs of two parts instead of three 159.
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
    gd_outputs_kernel(const __grid_constant__ Args g) {
  using K = OutCfg<T>;
  constexpr int DP = K::DP, PC = K::PC, NT = kOutThreads;
  extern __shared__ __align__(1024) unsigned char smem[];
  OutTab& tab = *reinterpret_cast<OutTab*>(smem + K::kTab);
  const GdArgs& a = g.a;
  const Place p = place_of(g, blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = (warp & 3) * 32 + lane, half = warp >> 2;
  T* o = static_cast<T*>(a.o) + p.b * a.ob + p.h * a.oh;
  float* o_part = a.o_part ? a.o_part + ((long long)p.b * a.H + p.h) * a.dvp : nullptr;
  const long long part_t = (long long)a.B * a.H * a.dvp;
  const int live = (int)(a.T - p.t0 < C ? a.T - p.t0 : C);  // rows of the tensor
  for (int i = tid; i < (live - p.n) * a.dvp; i += NT) {    // zeros past the length
    const long long t = p.t0 + p.n + i / a.dvp;
    if (o_part) o_part[t * part_t + i % a.dvp] = 0.f;
    else o[t * a.ot + i % a.dvp] = from_f32<T>(0.f);
  }
  if (p.n == 0) return;
  const int rows = 64 * g.dkt, cols = 64 * g.dvt;
  const float* S = g.S + p.slot * rows * cols;
  const T *q = rows_of<T>(a.q, p.t0, p.b, p.hq), *k = rows_of<T>(a.k, p.t0, p.b, p.hq);
  DataRows<T, C, 1, NT> qs, ks;
  QuadRows<64, 2, NT> ss;
  auto fetch = [&](int ct) {
    qs.fetch(q, a.q.st, 0, p.n, ct * 64, a.dk, 1);
    ks.fetch(k, a.k.st, 0, p.n, ct * 64, a.dk, 1);
    ss.fetch(S + ct * 64 * 4, rows, 64, g.dvt);
  };
  fetch(0);
  if (tid == 0) {
    ask_l2(g.E + p.at * C * cols, C * cols * 4);
    for (int c4 = 0; g.dkt > 1 && c4 < cols / 4; ++c4) ask_l2(S + (c4 * rows + 64) * 4, 64 * 16);
  }
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
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
      const int c0 = half * 64 + x * 16;
      float2 v[8];
      if ((c0 >> 5) <= (warp & 3)) read16(mine + c0, v);
      decayed<false>(v, row, c0, tab.gates);
      put16<PC>(smem, 2 * kTile, row, c0, v);
    }
  }
  const float up = tab.gates.up[row];
  for (int vt = 0; vt < g.dvt; ++vt) {
    es.template place<PC>(smem + K::kU, kTile, kTile, C, 1, tab.gates.beta);
    steps.run([&] {
      product<PC, PC, PC - 1>(tmem, k_major(base, 2 * kTile, kTile), mn_major(base + K::kU, kTile, kTile), 8,
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
      if (row >= p.n) continue;
      if (o_part) store16<float>(o_part + (p.t0 + row) * part_t + c0, a.dvp - c0, v);
      else store16<T>(o + (p.t0 + row) * a.ot + c0, a.dvp - c0, v);
    }
  }
  finish(tmem, 256, steps.ok, g.status);
}

template <typename K>
cudaError_t allow(K kernel, uint32_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

}  // namespace

namespace {
template <typename T, int NT>
cudaError_t prepare(const Args& g, bool keep_inverse, cudaStream_t s) {
  constexpr uint32_t smem = kPrepTab<NT> + sizeof(PrepTab);
  const cudaError_t e = allow(gd_prepare_kernel<T, NT>, smem);
  if (e != cudaSuccess) return e;
  gd_prepare_kernel<T, NT><<<grid_of(g, 512 / NT), NT, smem, s>>>(g, keep_inverse);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_prepare(const Args& g, bool keep_inverse, cudaStream_t s) {
  const bool few = 4LL * g.nbh * g.chunks <= 5LL * seq_sm_count();
  cudaError_t e = cudaSuccess;
  PRNN_BY_DTYPE(g.a.dtype, T, e = (few ? prepare<T, 512>(g, keep_inverse, s) : prepare<T, 256>(g, keep_inverse, s)));
  return e;
}

namespace {
template <int PK, bool REV, int SL>
cudaError_t chain(const Args& g, cudaStream_t s) {
  using K = ChainCfg<SL, PK, REV>;
  constexpr uint32_t smem = K::kTab + sizeof(ChainTab);
  const cudaError_t e = allow(gd_chain_kernel<PK, REV, SL>, smem);
  if (e != cudaSuccess) return e;
  gd_chain_kernel<PK, REV, SL><<<dim3(g.nbh, (g.a.dv + SL - 1) / SL), K::kThreads, smem, s>>>(g);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_chain(const Args& g, bool reverse, cudaStream_t s) {
  const bool narrow = g.a.dv <= 32 || (long long)g.nbh * ((g.a.dv + 31) / 32) <= seq_sm_count();
  cudaError_t e = cudaSuccess;
  PRNN_BY_DTYPE(g.a.dtype, T, {
    constexpr int PK = kData<T>;
    if (reverse) e = narrow ? chain<PK, true, 32>(g, s) : chain<PK, true, 64>(g, s);
    else e = narrow ? chain<PK, false, 32>(g, s) : chain<PK, false, 64>(g, s);
  });
  return e;
}

cudaError_t launch_outputs(const Args& g, cudaStream_t s) {
  PRNN_BY_DTYPE(g.a.dtype, T, {
    constexpr uint32_t smem = OutCfg<T>::kTab + sizeof(OutTab);
    const cudaError_t e = allow(gd_outputs_kernel<T>, smem);
    if (e != cudaSuccess) return e;
    gd_outputs_kernel<T><<<(unsigned)(g.nbh * g.chunks), kOutThreads, smem, s>>>(g);
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
  size_t one;                                       // of all for one head
};
// Heads go together in groups whose scratch stays within kMost bytes.
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
  p.one = w + k + gates + E + S + (backward ? inv + E + 2 * Z0 : 0);
  p.nbh = (int)std::min<size_t>((size_t)B * H, std::max<size_t>(1, kMost / p.one));
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

// A row of a head's values per warp: x [T][B][heads][d] with any strides into rows of dp >= d values, zeros behind d.
template <typename T>
__global__ void __launch_bounds__(256) gd_copy_kernel(const T* x, long long st, long long sb, long long sh, int B, int heads,
                                                      int d, int dp, long long rows, T* out) {
  const int lane = threadIdx.x & 31;
  for (long long row = blockIdx.x * 8LL + (threadIdx.x >> 5); row < rows; row += gridDim.x * 8LL) {
    const long long tb = row / heads, t = tb / B;
    const T* from = x + t * st + (tb - t * B) * sb + (row - tb * heads) * sh;
    for (int k = lane; k < dp; k += 32) out[row * dp + k] = k < d ? from[k] : from_f32<T>(0.f);
  }
}
// out[t][b][hq][0 .. d) = sum of the `group` heads of part [T][B][H][dp] that share hq.
template <typename T>
__global__ void __launch_bounds__(256) gd_join_kernel(const float* part, T* out, long long ot, long long ob, long long oh,
                                                      int B, int heads, int group, int d, int dp, long long rows) {
  const int lane = threadIdx.x & 31;
  for (long long row = blockIdx.x * 8LL + (threadIdx.x >> 5); row < rows; row += gridDim.x * 8LL) {
    const long long tb = row / heads, t = tb / B;
    T* to = out + t * ot + (tb - t * B) * ob + (row - tb * heads) * oh;
    const float* from = part + row * group * dp;
    for (int k = lane; k < d; k += 32) {
      float s = 0.f;
      for (int j = 0; j < group; ++j) s += from[(long long)j * dp + k];
      to[k] = from_f32<T>(s);
    }
  }
}

int up8(int d) { return (d + 7) / 8 * 8; }
// Rows of d values that 16-byte accesses fit.
bool packs(prnn_dtype_t dtype, const void* p, int d, int T, int B, int heads, long long t, long long b, long long h) {
  const int v = dtype == PRNN_F32 ? 4 : 8;
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && d % 8 == 0 && (T == 1 || t % v == 0) && (B == 1 || b % v == 0) &&
         (heads == 1 || h % v == 0);
}

// Tensors that the kernels cannot read or write in place: copies of the data, fp32 parts of the results.
struct Moves {
  struct In {
    LaSeq GdArgs::*seq;
    int heads, d;
    size_t bytes;
  } in[4];
  struct Out {
    void* out;
    long long t, b, h;
    int group, d;
    float* GdArgs::*part;
    size_t bytes;
  } out[3];
  int ins = 0, outs = 0;
  size_t total = 0;
};
Moves moves_of(const GdArgs& a, bool backward) {
  Moves m;
  const int hq = a.H / a.q.share;
  const size_t esz = a.dtype == PRNN_F32 ? 4 : 2, tokens = (size_t)a.T * a.B;
  auto in = [&](LaSeq GdArgs::*seq, int heads, int d) {
    const LaSeq& x = a.*seq;
    if (packs(a.dtype, x.p, d, a.T, a.B, heads, x.st, x.sb, x.sh)) return;
    m.in[m.ins++] = {seq, heads, d, up16(tokens * heads * up8(d) * esz)};
    m.total += m.in[m.ins - 1].bytes;
  };
  auto out = [&](void* p, long long t, long long b, long long h, int group, int d, float* GdArgs::*part) {
    if (!p || (group == 1 && packs(a.dtype, p, d, a.T, a.B, a.H, t, b, h))) return;
    m.out[m.outs++] = {p, t, b, h, group, d, part, up16(tokens * a.H * up8(d) * 4)};
    m.total += m.out[m.outs - 1].bytes;
  };
  in(&GdArgs::q, hq, a.dk);
  in(&GdArgs::k, hq, a.dk);
  in(&GdArgs::v, a.H, a.dv);
  if (!backward) {
    out(a.o, a.ot, a.ob, a.oh, 1, a.dv, &GdArgs::o_part);
    return m;
  }
  in(&GdArgs::d_o, a.H, a.dv);
  out(a.dq_out, a.dqt, a.dqb, a.dqh, a.q.share, a.dk, &GdArgs::dq_part);
  out(a.dk_out, a.dkt, a.dkb, a.dkh, a.q.share, a.dk, &GdArgs::dk_part);
  out(a.dv_out, a.dvt, a.dvb, a.dvh, 1, a.dv, &GdArgs::dv_part);
  return m;
}
unsigned blocks_for(long long rows) {
  return (unsigned)std::max(1LL, std::min((rows + 7) / 8, 16LL * seq_sm_count()));
}

}  // namespace

// Short sequences go token by token: that takes about 0.35 us a token and 1.8 ns more for each block of 16 columns, chunks
// about 40 us for the first (in the gradients four times the one, twice the other).  Measured, tokens by tokens
// and in chunks, us, bf16: 8 heads of 64 x 64, 64 tokens 22 and 31, 96 tokens 31 and 33, 128 tokens 40 and 33; 16 heads of
// 128 x 128, 64 tokens 29 and 40, 96 tokens 43 and 42; 128 heads, 16 tokens 32 and 55, 32 tokens 58 and 55; gradients of 8 heads of
// 64 x 64, 32 tokens 53 and 60, 48 tokens 71 and 60; of 128 heads of 128 x 128, 16 tokens 141 and 96.
bool gd_tc_serves(int T, int B, int H, int dk, int dv, bool backward) {
  const double blocks = (double)B * H * ((dv + 15) / 16);
  if (dk > 128 || dv > 128 || T * (200.0 + blocks) < (backward ? 11000.0 : 22000.0)) return false;
  // (a head of millions of tokens has too much scratch: it goes token by token as well)
  return plan_of(PRNN_F32, T, B, H, dk, dv, backward).one <= kMost;
}

size_t gd_tc_workspace(const GdArgs& a, bool backward) {
  return plan_of(a.dtype, a.T, a.B, a.H, a.dk, a.dv, backward).total + moves_of(a, backward).total;
}

cudaError_t launch_gd_tc(GdArgs a, void* scratch, bool backward, cudaStream_t s) {
  const Plan p = plan_of(a.dtype, a.T, a.B, a.H, a.dk, a.dv, backward);
  Args g{};
  g.chunks = p.chunks;
  g.dkt = p.dkt;
  g.dvt = p.dvt;
  g.status = seq_status_word();
  if (!g.status) return cudaErrorUnknown;
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
  const Moves m = moves_of(a, backward);
  a.dkp = up8(a.dk);
  a.dvp = up8(a.dv);
  a.o_part = a.dq_part = a.dk_part = a.dv_part = nullptr;
  for (int i = 0; i < m.ins; ++i) {
    const Moves::In& in = m.in[i];
    LaSeq& x = a.*in.seq;
    const int dp = up8(in.d);
    const long long n = (long long)a.T * a.B * in.heads;
    void* to = take(in.bytes);
    PRNN_BY_DTYPE(a.dtype, T, (gd_copy_kernel<T><<<blocks_for(n), 256, 0, s>>>(
        static_cast<const T*>(x.p), x.st, x.sb, x.sh, a.B, in.heads, in.d, dp, n, static_cast<T*>(to))));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    x = {to, (long long)a.B * in.heads * dp, (long long)in.heads * dp, dp, x.share};
  }
  for (int i = 0; i < m.outs; ++i) a.*m.out[i].part = take(m.out[i].bytes);
  g.a = a;
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
  for (int i = 0; i < m.outs; ++i) {
    const Moves::Out& o = m.out[i];
    const long long n = (long long)a.T * a.B * (a.H / o.group);
    PRNN_BY_DTYPE(a.dtype, T, (gd_join_kernel<T><<<blocks_for(n), 256, 0, s>>>(
        a.*o.part, static_cast<T*>(o.out), o.t, o.b, o.h, a.B, a.H / o.group, o.group, o.d, up8(o.d), n)));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace prnn
