// linear_attention_tc.cu -- the `mix` operation of seq_internal.h on the 5th-generation tensor
// cores, for fp16 and bf16 data: linear attention's forward pass and all three products of its
// backward pass.
//
// A CTA walks the chunks of C tokens of one (role, sequence, head) and 64 of the e columns, the
// state in registers.  With l the decay, per chunk entered with state X:
//   P  = A B^T            (C x C, scores)             tcgen05, operands K-major
//   O1 = (P o D) C        D_ij = l^|i-j|, causal      P goes back to TMEM as the A operand
//   O2 = A X                                          X in shared memory, MN-major
//   U  = B^T (w C)        w_j the tokens' decays      B is the same tile, MN-major
//   out_i = s_intra O1_i + s_inter l^(.) O2_i,   X <- l^n X + s_add U.
// One TMA load of a tile serves both majors, so nothing is transposed.  Every power of l has an
// exponent >= 0 (D in blocks of 16 columns: l^(i-j) = l^(i-j0-15) l^(15-(j-j0))), so no decay
// overflows.
//
// Rounding.  The products take 16-bit operands.  The data enters as it is; what is computed in between
// enters as a sum of parts of the data's type: P and X in two (bf16: 16 bits; their error stays far
// below the output's one rounding), w C in two for fp16 (22 bits), and for bf16 in three (24 bits)
// where the fp32 state is an output and two where it only feeds 16-bit ones.  All products accumulate
// in fp32.  For fp16, whose range would not hold them, P is scaled by a power of two per row (its largest
// weighted score) and X and w C per tile, taken back after the product.  A value 2^27 and more below the largest
// finite one of its tile keeps fewer bits than a 16-bit output has; a scale per column would need
// the columns' maxima over all tokens before the first could be stored.
//
// Warps: 0 loads (TMA), 1 and 2 issue the matrix products, 4-11 turn scores into operands (a row per
// thread, every other block of 16 columns), 12-19 own the state (a row of X and half the columns),
// 20-27 make w C and write the output (a row and half the columns).  The tensor cores run U(c), O2(c),
// P(c+1) and O1(c) while the state is updated, the next chunk's w C made, its scores weighted and the
// last output written; each tile of chunk c + 2 is requested as the last product that reads chunk c's
// ends. The two parts of X stand side by side in one product (N = 128), which reads Q once.
//
// What bounds it: memory would take 40 us for T = 8192, 2 sequences of 16 heads of 128 x 128 bf16, and the
// kernel takes 127.  A chunk of 112 tokens costs a CTA about 4600 cycles: the products read 280 KB of
// operands from shared memory, TMA and the warps move 190 KB more (3600 cycles at 128 bytes each), and the
// chain w C -> U -> X -> O2 with its barriers is about as long.  C = 112 is what two chunks in flight
// leave room for at 128 x 128; 96 took 136 us, 80 with three chunks in flight 152 (112 took 130 then).  Other figures,
// us: T = 2048, 4 sequences 52; at 64 x 64 37; T = 256, 32 sequences 96; gradients of T = 2048, 4 sequences 136.
// fp16 takes 145, 61, 41, 99 and 176 for its maxima.
// The CUDA-core kernel of the first version took 10353 for the first of these.
#include <cuda.h>

#include <algorithm>
#include <cstdint>

#include "linear_attention_plan.h"
#include "linear_attention_tables.h"
#include "seq_common.cuh"
#include "seq_internal.h"
#include "seq_tc.cuh"

namespace prnn {
namespace {

using namespace tc;

constexpr int kThreads = 896, kSlice = 64, kHalfSlice = 32;
constexpr uint32_t kTmemCols = 512;
// columns of tensor memory: two score tiles, O1, O2 (a part of X each), U
constexpr uint32_t kColP = 0, kColO1 = 256, kColO2 = 320, kColU = 448;

template <typename T, int DB, int PARTS>
struct Cfg {
  static constexpr int C = DB == 2 ? 112 : 128;  // tokens per chunk: what the rings leave room for
  static constexpr int kParts = PARTS;           // of w C
  static constexpr uint32_t kBlock = C * 128;    // one [C][64] tile, 128-byte swizzled
  static constexpr uint32_t kStage = (2 * DB + 1) * kBlock;
  static constexpr uint32_t kStateTile = DB * 64 * 128;
  static constexpr uint32_t oW = 2 * kStage;     // w C, kParts tiles
  static constexpr uint32_t oX = oW + kParts * kBlock;  // X, two tiles
  static constexpr uint32_t oTab = oX + 2 * kStateTile;
};

struct TcRole {
  int ia, ib, ic;     // tensor maps of a, b, c
  int sa, sb, sc;     // heads sharing one
  void* out;
  long long ot, ob, oh;
  int form, d, e;     // how the output is stored (OutForm)
  const float* x0;
  float* x_end;
  int x_t, rev, lead;
  float s_intra, s_inter, s_add;
};
struct TcArgs {
  TcRole role[3];
  int T, B, H;
  const float* log_decay;
  const int32_t* lens;
  int* status;
  // segments: cps chunks each; states of `subs` runs of cpb chunks in part
  int segs, cps, subs, cpb, slices, states_only;
  float* part;        // [role][B*H][subs][slices * 64][128]
};
struct Maps {
  CUtensorMap m[4];
};

// A from tensor memory
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                        uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                         int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ float top_of(float top, float2 v) { return fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y))); }
// The same of the finite values alone (v + 0 v is NaN for an infinity, which fmaxf passes over).  A scale is theirs:
// an infinity is to reach the outputs as what it is, and not to take the bits of the numbers that share its
// scale.  It is looked for only where the plain maximum is one (T = 8192, 2 sequences of 16 heads of 128 x 128: 145 us;
// 148 with it looked for in every maximum).
__device__ __forceinline__ float finite_top(float top, float2 v) { return top_of(top, fma2(v, both(0.f), v)); }
__device__ __forceinline__ bool infinite(float top) { return top > 3.4028235e38f; }
// 2^k such that max * 2^k lies in [2^13, 2^14), for 0 <= max < infinity; and 2^-k.
__device__ __forceinline__ float2 fit_scale(float max) {
  int k = 13 + 127 - (int)(__float_as_uint(max) >> 23);
  k = k > 100 ? 100 : k;
  return make_float2(__uint_as_float((uint32_t)(127 + k) << 23), __uint_as_float((uint32_t)(127 - k) << 23));
}
// The largest of 256 threads' values (warps w = 0..7 of a group with named barrier id).
__device__ __forceinline__ float group_max(float v, float* red, int w, int id) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory");
  if ((threadIdx.x & 31) == 0) red[w] = v;
  asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory");
  float m = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
  return m;
}

// 32 columns of one row at p, of which the first m are the output's.
enum OutForm { kOutPacked = 0, kOutF32 = 1, kOutSingle = 2 };  // kOutSingle: value by value (| kOutF32)
template <typename T>
__device__ __forceinline__ void store_out(char* p, int form, int m, const float2 (&v)[kHalfSlice / 2]) {
  if (form == kOutPacked) {
    uint4* to = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int q = 0; q < kHalfSlice / 8; ++q)
      if (8 * q < m) {
        float2 k[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        uint4 u;
        u.x = take<T>(k[0]);
        u.y = take<T>(k[1]);
        u.z = take<T>(k[2]);
        u.w = take<T>(k[3]);
        to[q] = u;
      }
  } else if (form == kOutF32) {
    float4* to = reinterpret_cast<float4*>(p);
#pragma unroll
    for (int q = 0; q < kHalfSlice / 4; ++q)
      if (4 * q < m) to[q] = make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
  } else {
#pragma unroll
    for (int j = 0; j < kHalfSlice; ++j)
      if (j < m) {
        const float f = j & 1 ? v[j / 2].y : v[j / 2].x;
        if (form & kOutF32)
          reinterpret_cast<float*>(p)[j] = f;
        else
          reinterpret_cast<T*>(p)[j] = from_f32<T>(f);
      }
  }
}

// The state's rows start on 16 bytes and are not transposed.
__device__ __forceinline__ bool rows_of_4(const TcRole& r, const float* p) {
  return !r.x_t && r.e % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <typename T, int DB, int PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    la_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TcArgs g) {
  using K = Cfg<T, DB, PARTS>;
  constexpr int C = K::C;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  extern __shared__ __align__(1024) unsigned char smem[];
  Tables& tab = *reinterpret_cast<Tables*>(smem + K::oTab);
  const TcRole& r = g.role[blockIdx.y];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int slice = blockIdx.x % g.slices, seg = blockIdx.x / g.slices % (g.states_only ? g.subs : g.segs);
  const int bh = blockIdx.x / g.slices / (g.states_only ? g.subs : g.segs), b = bh / g.H, h = bh % g.H;
  const int e0 = slice * kSlice;
  if (e0 >= r.e) return;
  int len = g.T;
  if (g.lens) {
    len = g.lens[b];
    len = len < 0 ? 0 : (len > g.T ? g.T : len);
  }
  const int chunks = (len + C - 1) / C;
  // this CTA's run of chunks, in the order of processing
  const int per = g.states_only ? g.cpb : g.cps;
  const int from = min(seg * per, chunks), to = min((seg + 1) * per, chunks), nc = to - from;
  const float ld = g.log_decay[h];
  const int last = len - (chunks - 1) * C;  // tokens of the last chunk
  auto chunk_of = [&](int c) { return r.rev ? chunks - 1 - c : c; };
  auto tokens_of = [&](int c) { return chunk_of(c) == chunks - 1 ? last : C; };
  // tokens processed before chunk c of the order
  auto before = [&](int c) {
    if (c <= 0) return 0;
    if (c >= chunks) return len;
    return r.rev ? last + (c - 1) * C : c * C;
  };
  const bool writes_end = !g.states_only && r.x_end && (nc > 0 ? to == chunks : (chunks == 0 && seg == 0));

  const int osize = r.form & kOutF32 ? 4 : (int)sizeof(T);
  if (!g.states_only && r.out) {  // zeros past the length
    const int ncol = min(kSlice, r.e - e0);
    for (int c = max(seg * per, chunks); c < (seg + 1) * per && c * C < g.T; ++c) {
      const int rows = min(C, g.T - c * C);
      const float2 z[kHalfSlice / 2] = {};
      for (int i = tid; i < rows * 2; i += kThreads) {
        const int row = i / 2, q = i % 2 * kHalfSlice;
        store_out<T>(static_cast<char*>(r.out) + ((c * C + row) * r.ot + b * r.ob + h * r.oh + e0 + q) * osize,
                     r.form, ncol - q, z);
      }
    }
  }
  if (nc == 0 && !writes_end) return;

  const bool with_out = !g.states_only;
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {  // the swizzled tiles need it; no static shared memory precedes them
    if (tid == 0) atomicExch(g.status, 1);
    return;
  }
  // The loads of one chunk: b and a (scores, state), then c.
  const int db = (r.d + 63) / 64;
  auto load_b = [&](int c) {
    const int s = c & 1, t0 = chunk_of(from + c) * C;
    const uint32_t at = base + s * K::kStage + DB * K::kBlock;
    mbar_arrive_expect_tx(&tab.ab_full[s], (with_out ? 2 : 1) * db * K::kBlock);
    for (int k = 0; k < db; ++k)
      tma_load(at + k * K::kBlock, &maps.m[r.ib], &tab.ab_full[s], k * 64, h / r.sb, b, t0);
  };
  auto load_a = [&](int c) {
    const int s = c & 1, t0 = chunk_of(from + c) * C;
    for (int k = 0; k < db; ++k)
      tma_load(base + s * K::kStage + k * K::kBlock, &maps.m[r.ia], &tab.ab_full[s], k * 64, h / r.sa, b, t0);
  };
  auto load_c = [&](int c) {
    const int s = c & 1, t0 = chunk_of(from + c) * C;
    mbar_arrive_expect_tx(&tab.c_full[s], K::kBlock);
    tma_load(base + s * K::kStage + 2 * DB * K::kBlock, &maps.m[r.ic], &tab.c_full[s], e0, h / r.sc, b, t0);
  };
  // The first two chunks are requested before anything else is set up.
  if (warp == 0 && elected()) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tab.ab_full[i], 1);
      mbar_init(&tab.c_full[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int c = 0; c < min(nc, 2); ++c) {
      load_b(c);
      if (with_out) load_a(c);
      load_c(c);
    }
  }
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tab.a_free[i], 2);
      mbar_init(&tab.b_free[i], with_out ? 2 : 1);
      mbar_init(&tab.c_free[i], 1);
      mbar_init(&tab.p_full[i], 1);
      mbar_init(&tab.p_ready[i], 8);
      mbar_init(&tab.w_ready[i], 8);
    }
    mbar_init(&tab.o_full, 1);
    mbar_init(&tab.o_free, 8);
    mbar_init(&tab.o2_full, 1);
    mbar_init(&tab.o2_free, 8);
    mbar_init(&tab.x_ready, 8);
    mbar_init(&tab.u_full, 1);
    mbar_init(&tab.u_free, 8);
    mbar_init(&tab.done, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tab.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  if (tid < 132) tab.pw[tid] = decay_pow(ld, tid);
  else if (tid < 148) tab.dec[tid - 132] = decay_pow(ld, r.rev ? tid - 132 : 147 - tid);
  for (int i = warp; i < 32; i += kThreads / 32) {
    const int gap = r.rev ? lane - i : i - lane;
    tab.diag[i][lane] = gap >= 0 ? decay_pow(ld, gap) : 0.f;
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tmem = tab.tmem;
  // a state enters the first chunk unless it is known to be zero
  const bool enters = r.x0 != nullptr || (seg > 0 && !g.states_only);
  // A wait that runs out is remembered and the work goes on (every later wait then ends at once):
  // no thread leaves the others waiting, and nothing is left in flight.
  bool ok = true;
  auto wait = [&](uint64_t* bar, int turn) { seq_wait(bar, turn & 1, ok); };
  auto warp_wait = [&](uint64_t* bar, int turn) {
    wait(bar, turn);
    __syncwarp();
  };

  if (warp == 0) {
    if (elected()) {
      // ---- loads: each tile as soon as the products that read the one before it have ended ----
      for (int c = 2; c < nc; ++c) {
        const int s = c & 1, turn = (c >> 1) - 1;
        wait(&tab.b_free[s], turn);
        load_b(c);
        if (with_out) {
          wait(&tab.a_free[s], turn);
          load_a(c);
        }
        wait(&tab.c_free[s], turn);
        load_c(c);
      }
      for (int c = max(0, nc - 2); c < nc; ++c) {  // every load lands before the CTA leaves
        bool landed = true;  // with a limit of its own, whatever has run out before
        seq_wait(&tab.ab_full[c & 1], (c >> 1) & 1, landed);
        seq_wait(&tab.c_full[c & 1], (c >> 1) & 1, landed);
        ok = ok && landed;
      }
    }
  } else if (warp == 1 || warp == 2) {
    // ---- matrix products: warp 1 those of the state (U, O2), warp 2 those of the scores (P, O1), so that
    // one's waits run under the other's products.  A product costs its thread as few instructions as can be:
    // descriptors are made once and stepped by constants ----
    if (elected()) {
      const int dsteps = (r.d + 15) / 16;
      const uint64_t da0 = sw128_kmajor_desc(base), db0 = sw128_kmajor_desc(base + DB * K::kBlock);
      constexpr uint64_t stage = K::kStage >> 4;
      constexpr auto kstep = [](int k) { return (uint64_t)(((k / 4) * K::kBlock + (k % 4) * 32) >> 4); };
      if (warp == 1) {
        const uint64_t dbt0 = mn_desc(base + DB * K::kBlock, K::kBlock);
        const uint64_t dw = mn_desc(base + K::oW, 1024), dx = mn_desc(base + K::oX, K::kStateTile);
        for (int c = 0; c < nc; ++c) {
          const uint64_t off = (c & 1) * stage;
          wait(&tab.ab_full[c & 1], c >> 1);
          wait(&tab.w_ready[c & 1], c >> 1);
          if (c > 0) wait(&tab.u_free, c - 1);
          after_sync();
          const uint64_t dbt = here(dbt0 + off), dwc = here(dw);
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int k = 0; k < C / 16; ++k)  // 16 tokens = 2048 bytes = 128 units
              umma_f16(tmem + kColU, dbt + 128 * k, dwc + (PARTS - 1 - p) * (K::kBlock >> 4) + 128 * k,
                       idesc<T>(128, kSlice) | kAMn | kBMn, p > 0 || k > 0);
          umma_commit(&tab.u_full);
          umma_commit(&tab.b_free[c & 1]);
          if (!with_out) {
            umma_commit(&tab.c_free[c & 1]);
            continue;
          }
          if (c > 0 || enters) {
            const int turn = enters ? c : c - 1;
            wait(&tab.x_ready, turn);
            if (turn > 0) wait(&tab.o2_free, turn - 1);
            after_sync();
            const uint64_t da = here(da0 + off), dxc = here(dx);
#pragma unroll
            for (int k = 0; k < 4 * DB; ++k)
              if (k < dsteps)
                umma_f16(tmem + kColO2, da + kstep(k), dxc + 128 * k, idesc<T>(128, 2 * kSlice) | kBMn, k > 0);
            umma_commit(&tab.o2_full);
          }
          umma_commit(&tab.a_free[c & 1]);
        }
      } else if (with_out) {
        const uint64_t dc0 = mn_desc(base + 2 * DB * K::kBlock, 1024);
        auto qk = [&](int c) {
          wait(&tab.ab_full[c & 1], c >> 1);
          after_sync();
          const uint64_t da = here(da0 + (c & 1) * stage), db = here(db0 + (c & 1) * stage);
          const uint32_t d = tmem + kColP + (c & 1) * 128;
#pragma unroll
          for (int k = 0; k < 4 * DB; ++k)
            if (k < dsteps) umma_f16(d, da + kstep(k), db + kstep(k), idesc<T>(128, C), k > 0);
          umma_commit(&tab.p_full[c & 1]);
          umma_commit(&tab.a_free[c & 1]);
          umma_commit(&tab.b_free[c & 1]);
        };
        if (nc > 0) qk(0);
        for (int c = 0; c < nc; ++c) {
          if (c + 1 < nc) qk(c + 1);
          wait(&tab.c_full[c & 1], c >> 1);
          wait(&tab.w_ready[c & 1], c >> 1);  // rows of C past the length have been cleared
          wait(&tab.p_ready[c & 1], c >> 1);
          if (c > 0) wait(&tab.o_free, c - 1);
          after_sync();
          const uint32_t pa = tmem + kColP + (c & 1) * 128, d = tmem + kColO1;
          const uint64_t dc = here(dc0 + (c & 1) * stage);
#pragma unroll
          for (int k = 0; k < C / 16; ++k) {
            umma_ts(d, pa + 16 * k, dc + 128 * k, idesc<T>(128, kSlice) | kBMn, k > 0);
            umma_ts(d, pa + 16 * k + 8, dc + 128 * k, idesc<T>(128, kSlice) | kBMn, 1);
          }
          umma_commit(&tab.o_full);
          umma_commit(&tab.c_free[c & 1]);
        }
      }
      // every product has read its operands before the CTA leaves
      umma_commit(&tab.done);
      bool read = true;
      seq_wait(&tab.done, 0, read);
      ok = ok && read;
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- scores to operands: row i of P, blocks of 16 columns half, half + 2, ... ----
    const int w = (warp - 4) & 3, half = (warp - 4) >> 2, i = w * 32 + lane;
    const uint32_t quad = (uint32_t)(w * 32) << 16;
    const bool rev = r.rev;
    for (int c = 0; c < (with_out ? nc : 0); ++c) {
      warp_wait(&tab.p_full[c & 1], c >> 1);
      after_sync();
      const uint32_t at = tmem + quad + kColP + (c & 1) * 128;
      const int n = tokens_of(from + c);
      // columns [16 jb, 16 jb + 16) against this warp's rows [32 w, 32 w + 32)
      auto nothing = [&](int jb) { return rev ? jb < 2 * w : jb > 2 * w + 1; };
      // this row's scores of block jb, weighted with their decays; 0 behind the mask and past the length, where a
      // score may be anything
      auto weighted = [&](int jb, float2 (&v)[8]) {
        uint32_t raw[16];
        tmem_ld16(at + 16 * jb, raw);
        const bool diagonal = (jb >> 1) == w;
        const float* dec = diagonal ? tab.diag[lane] + (jb & 1) * 16 : tab.dec;
        const float2 f = both(diagonal ? 1.f : tab.pw[rev ? 16 * jb - i : i - 16 * jb - 15]);
        wait_ld();
        if (16 * jb + 16 > n)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (16 * jb + j >= n) raw[j] = 0u;
        if (diagonal) {
          const int gap = rev ? i - 16 * jb : 16 * jb + 15 - i;  // in reverse the first `gap` columns, else the last
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((rev ? j : 15 - j) < gap) raw[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 d = *reinterpret_cast<const float4*>(dec + 2 * j);
          v[j] = mul2(pair_at(raw, j), mul2(f, make_float2(d.x, d.y)));
          v[j + 1] = mul2(pair_at(raw, j + 1), mul2(f, make_float2(d.z, d.w)));
        }
      };
      float2 scale = both(1.f);
      if constexpr (kHalf) {
        // The row's scale fits its largest weighted score, so only what the row sums counts: a score behind
        // the mask or one that has long decayed may be 2^30 times the others and would leave them no
        // bits.  The weighted scores go back to tensor memory, which is cheaper than weighting them twice (gradients
        // of T = 2048, 4 sequences of 16 heads of 128 x 128: 172 us, weighted twice 190).
        float top = 0.f;
#pragma unroll 1
        for (int jb = half; jb < C / 16; jb += 2) {
          if (nothing(jb)) continue;
          float2 v[8];
          weighted(jb, v);
          uint32_t raw[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            top = top_of(top, v[j]);
            raw[2 * j] = __float_as_uint(v[j].x);
            raw[2 * j + 1] = __float_as_uint(v[j].y);
          }
          tmem_st16(at + 16 * jb, raw);
        }
        wait_st();
        if (__any_sync(0xffffffffu, infinite(top))) {
          top = 0.f;
#pragma unroll 1
          for (int jb = half; jb < C / 16; jb += 2) {
            if (nothing(jb)) continue;
            uint32_t raw[16];
            tmem_ld16(at + 16 * jb, raw);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) top = finite_top(top, pair_at(raw, j));
          }
        }
        tab.row_top[half][i] = top;
        asm volatile("bar.sync 3, 256;" ::: "memory");
        const float2 f = fit_scale(fmaxf(tab.row_top[0][i], tab.row_top[1][i]));
        asm volatile("bar.sync 3, 256;" ::: "memory");
        scale = both(f.x);
        if (half == 0) tab.row_scale[c & 3][i] = f.y;  // read by the output warps, after p_ready and o_full
      }
#pragma unroll 1
      for (int jb = half; jb < C / 16; jb += 2) {
        uint32_t o[16];
        if (nothing(jb)) {
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = 0u;
          tmem_st16(at + 16 * jb, o);
          continue;
        }
        float2 v[8];
        if constexpr (kHalf) {
          tmem_ld16(at + 16 * jb, o);
          wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mul2(pair_at(o, j), scale);
        } else {
          weighted(jb, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = take<T>(v[j]);
          o[8 + j] = take<T>(v[j]);
        }
        tmem_st16(at + 16 * jb, o);
      }
      wait_st();
      before_sync();
      warp_arrive(&tab.p_ready[c & 1]);
    }
  } else if (warp >= 12 && warp < 20) {
    // ---- the state: row `row` of X, columns [32 half, 32 half + 32) of the slice ----
    const int w = warp - 12, row = (w & 3) * 32 + lane, half = w >> 2;
    const uint32_t from_tmem = tmem + ((uint32_t)((w & 3) * 32) << 16) + kColU + half * kHalfSlice;
    const int col0 = e0 + half * kHalfSlice, ncol = min(kHalfSlice, r.e - col0);
    const size_t head = (size_t)bh * r.d * r.e;
    float2 X[kHalfSlice / 2];
#pragma unroll
    for (int j = 0; j < kHalfSlice / 2; ++j) X[j] = both(0.f);
    const int done_before = before(from);
    if (r.x0 && !g.states_only && row < r.d) {
      const float f = decay_pow(ld, done_before);
      const float* p = r.x0 + head + (r.x_t ? (size_t)col0 * r.d + row : (size_t)row * r.e + col0);
      const int step = r.x_t ? r.d : 1;
      if (rows_of_4(r, r.x0) && ncol == kHalfSlice) {
#pragma unroll
        for (int j = 0; j < kHalfSlice / 4; ++j) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p) + j);
          X[2 * j] = make_float2(f * v.x, f * v.y);
          X[2 * j + 1] = make_float2(f * v.z, f * v.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kHalfSlice / 2; ++j) {
          if (2 * j < ncol) X[j].x = f * p[2 * j * step];
          if (2 * j + 1 < ncol) X[j].y = f * p[(2 * j + 1) * step];
        }
      }
    }
    float* part = g.part + ((((size_t)blockIdx.y * g.B * g.H + bh) * g.subs * g.slices + slice) * kSlice +
                            half * kHalfSlice) * 128 + row;
    const size_t sub_size = (size_t)g.slices * kSlice * 128;
    if (!g.states_only) {
      const int subs = min(seg * (g.cps / g.cpb), (chunks + g.cpb - 1) / g.cpb);
      for (int u = 0; u < subs; ++u) {
        const float2 f = both(decay_pow(ld, done_before - before((u + 1) * g.cpb)));
        const float* p = part + u * sub_size;
#pragma unroll
        for (int j = 0; j < kHalfSlice / 2; ++j)
          X[j] = fma2(make_float2(__ldcg(p + 2 * j * 128), __ldcg(p + (2 * j + 1) * 128)), f, X[j]);
      }
    }
    unsigned char* tile = smem + K::oX + row * 128;
    auto publish = [&](int turn) {  // X as parts in shared memory, for the chunk of this turn
      float2 scale = both(1.f);
      if constexpr (kHalf) {
        float top = 0.f;
        if (row < r.d)
#pragma unroll
          for (int j = 0; j < kHalfSlice / 2; ++j) top = top_of(top, X[j]);
        top = group_max(top, tab.red[0], w, 1);
        if (infinite(top)) {  // the same for the whole group
          top = 0.f;
          if (row < r.d)
#pragma unroll
            for (int j = 0; j < kHalfSlice / 2; ++j) top = finite_top(top, X[j]);
          top = group_max(top, tab.red[0], w, 1);
        }
        const float2 f = fit_scale(top);
        scale = both(f.x);
        if (row == 0 && half == 0) tab.x_scale[turn & 1] = f.y;
      }
      if (row < db * 64) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 v = X[4 * q + j];
            if (kHalf) v = mul2(v, scale);
            hi[j] = take<T>(v);
            lo[j] = take<T>(v);
          }
          const uint32_t at = (uint32_t)(((half * 4 + q) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(tile + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(tile + K::kStateTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      to_async();
      warp_arrive(&tab.x_ready);
    };
    if (enters && with_out && nc > 0) publish(0);
    const float s_add = r.s_add;
    for (int c = 0; c < nc; ++c) {
      const float2 f = both(tab.pw[tokens_of(from + c)]);
      warp_wait(&tab.u_full, c);
      after_sync();
      const float2 s = both(s_add * (kHalf ? tab.w_scale[c & 3] : 1.f));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t u[16];
        tmem_ld16(from_tmem + 16 * q, u);
        wait_ld();
        if (q == 1) {
          before_sync();
          warp_arrive(&tab.u_free);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          X[8 * q + j] = fma2(make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), s,
                              mul2(f, X[8 * q + j]));
      }
      if (with_out && c + 1 < nc) {
        // the product with the state before has read its tile (there was one unless none entered)
        if (c > 0 || enters) warp_wait(&tab.o2_full, enters ? c : c - 1);
        publish(c + 1);
      }
    }
    if (writes_end && row < r.d) {
      float* p = r.x_end + head + (r.x_t ? (size_t)col0 * r.d + row : (size_t)row * r.e + col0);
      const int step = r.x_t ? r.d : 1;
      if (rows_of_4(r, r.x_end) && ncol == kHalfSlice) {
#pragma unroll
        for (int j = 0; j < kHalfSlice / 4; ++j)
          reinterpret_cast<float4*>(p)[j] = make_float4(X[2 * j].x, X[2 * j].y, X[2 * j + 1].x, X[2 * j + 1].y);
      } else {
#pragma unroll
        for (int j = 0; j < kHalfSlice / 2; ++j) {
          if (2 * j < ncol) p[2 * j * step] = X[j].x;
          if (2 * j + 1 < ncol) p[(2 * j + 1) * step] = X[j].y;
        }
      }
    }
    if (g.states_only) {
#pragma unroll
      for (int j = 0; j < kHalfSlice / 2; ++j) {
        part[seg * sub_size + 2 * j * 128] = X[j].x;
        part[seg * sub_size + (2 * j + 1) * 128] = X[j].y;
      }
    }
  } else if (warp >= 20) {
    // ---- w C: row i of the tile, decayed to the chunk's end; output: row i.  Columns [32 half, 32 half + 32)
    // of the slice ----
    const int w = warp - 20, half = w >> 2, i = (w & 3) * 32 + lane;
    const uint32_t from_tmem = tmem + ((uint32_t)((w & 3) * 32) << 16) + half * kHalfSlice;
    const int col0 = e0 + half * kHalfSlice, ncol = r.e - col0;
    // what every chunk needs of the role, taken from the parameters once
    const bool rev = r.rev;
    const int form = r.form, lead = r.lead;
    const float s_intra = r.s_intra, s_inter = r.s_inter;
    const long long row_bytes = r.ot * osize;
    char* const out = r.out ? static_cast<char*>(r.out) + (b * r.ob + h * r.oh + col0) * osize + i * row_bytes : nullptr;
    auto decayed = [&](int c) {
      const int n = tokens_of(from + c);
      warp_wait(&tab.c_full[c & 1], c >> 1);
      unsigned char* tile = smem + (c & 1) * K::kStage + 2 * DB * K::kBlock + i * 128;
      const int gap = (rev ? i : n - 1 - i) + 1 - lead;
      const float wj = i < n ? tab.pw[gap] : 0.f;
      uint32_t raw[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < n) v = *reinterpret_cast<const uint4*>(tile + (((half * 4 + q) ^ (i & 7)) << 4));
        raw[q][0] = v.x;
        raw[q][1] = v.y;
        raw[q][2] = v.z;
        raw[q][3] = v.w;
      }
      float2 f = both(wj);
      if constexpr (kHalf) {
        float top = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = top_of(top, unpack<T>(raw[q][k]));
        top = group_max(top * wj, tab.red[1], w, 2);
        if (infinite(top)) {
          top = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) top = finite_top(top, unpack<T>(raw[q][k]));
          top = group_max(top * wj, tab.red[1], w, 2);
        }
        const float2 s = fit_scale(top);
        f = mul2(f, both(s.x));
        if (i == 0 && half == 0) tab.w_scale[c & 3] = s.y;
      }
      if (c > 0) warp_wait(&tab.u_full, c - 1);
      if (n < C) {
        // Rows past the length may hold anything: the scores, which read them, are made first, then
        // they are cleared, so that 0 * anything stays 0.
        if (with_out) warp_wait(&tab.p_full[c & 1], c >> 1);
        else warp_wait(&tab.ab_full[c & 1], c >> 1);
        if (i >= n && i < C && half == 0) {
          const uint4 z = make_uint4(0, 0, 0, 0);
          for (int q = 0; q < 8; ++q) {
            *reinterpret_cast<uint4*>(tile + (q << 4)) = z;
            for (int k = 0; k < db; ++k)
              *reinterpret_cast<uint4*>(smem + (c & 1) * K::kStage + (DB + k) * K::kBlock + i * 128 + (q << 4)) = z;
          }
        }
      }
      if (i < C)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[K::kParts][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 v = mul2(unpack<T>(raw[q][k]), f);
#pragma unroll
            for (int m = 0; m < K::kParts; ++m) p[m][k] = take<T>(v);
          }
#pragma unroll
          for (int m = 0; m < K::kParts; ++m)
            *reinterpret_cast<uint4*>(smem + K::oW + m * K::kBlock + i * 128 + (((half * 4 + q) ^ (i & 7)) << 4)) =
                make_uint4(p[m][0], p[m][1], p[m][2], p[m][3]);
        }
      to_async();
      warp_arrive(&tab.w_ready[c & 1]);
    };
    auto output = [&](int c) {
      const int n = tokens_of(from + c), t0 = chunk_of(from + c) * C;
      float2 v[kHalfSlice / 2];
#pragma unroll
      for (int j = 0; j < kHalfSlice / 2; ++j) v[j] = both(0.f);
      if (c > 0 || enters) {
        warp_wait(&tab.o2_full, enters ? c : c - 1);
        after_sync();
        const int gap = (rev ? n - 1 - i : i) + lead;
        const float2 fx = both(s_inter * tab.pw[gap < 0 ? 0 : gap] * (kHalf ? tab.x_scale[c & 1] : 1.f));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t x[16], y[16];
          tmem_ld16(from_tmem + kColO2 + 16 * q, x);
          tmem_ld16(from_tmem + kColO2 + kSlice + 16 * q, y);
          wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[8 * q + j] = mul2(add2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])),
                                     make_float2(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]))), fx);
        }
        before_sync();
        warp_arrive(&tab.o2_free);
      }
      warp_wait(&tab.o_full, c);
      after_sync();
      const float2 fi = both(s_intra * (kHalf ? tab.row_scale[c & 3][i] : 1.f));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t a[16];
        tmem_ld16(from_tmem + kColO1 + 16 * q, a);
        wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[8 * q + j] = fma2(make_float2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1])), fi,
                              v[8 * q + j]);
      }
      before_sync();
      warp_arrive(&tab.o_free);
      if (i >= n)
#pragma unroll
        for (int j = 0; j < kHalfSlice / 2; ++j) v[j] = both(0.f);
      if (i < C && t0 + i < g.T && out) store_out<T>(out + t0 * row_bytes, form, ncol, v);
      __syncwarp();
    };
    if (nc > 0) decayed(0);
    for (int c = 0; c < nc; ++c) {
      if (c + 1 < nc) decayed(c + 1);
      if (with_out) output(c);
    }
  }
  if (!ok) atomicExch(g.status, 1);
  before_sync();
  __syncthreads();
  if (warp == 3) {
    after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// x [T][B][heads][d] with any strides into rows of dp >= d values, zeros behind d.
__global__ void __launch_bounds__(256) la_copy_kernel(const uint16_t* x, long long st, long long sb,
                                                      long long sh, int B, int heads, int d, int dp,
                                                      long long rows, uint16_t* out) {
  const long long n = rows * dp;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long row = i / dp;
    const int k = (int)(i - row * dp), h = (int)(row % heads);
    const long long tb = row / heads;
    out[i] = k < d ? x[tb / B * st + tb % B * sb + h * sh + k] : (uint16_t)0;
  }
}

// A sequence tensor as {d, heads, B, T}, read in boxes of 64 values of C tokens of one head.
bool encode(CUtensorMap* map, const LaSeq& x, int d, int heads, int B, int T, int C, bool half) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)B, (cuuint64_t)T};
  // the stride of an axis of one is never used, but has to be a legal one
  const cuuint64_t strides[3] = {(cuuint64_t)(heads > 1 ? x.sh * 2 : 16), (cuuint64_t)(B > 1 ? x.sb * 2 : 16),
                                 (cuuint64_t)(T > 1 ? x.st * 2 : 16)};
  const cuuint32_t box[4] = {64, 1, 1, (cuuint32_t)C}, estr[4] = {1, 1, 1, 1};
  return fn(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(x.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool axis_ok(long long stride, int n) {
  return n <= 1 || (stride > 0 && stride % 8 == 0 && stride < (1LL << 38));
}
bool seq_fits(const LaSeq& s, const LaArgs& a, int d) {
  return (reinterpret_cast<uintptr_t>(s.p) & 15) == 0 && d % 8 == 0 && axis_ok(s.st, a.T) &&
         axis_ok(s.sb, a.B) && axis_ok(s.sh, a.H / s.share);
}

constexpr size_t kStateBytes = kSlice * 128 * sizeof(float);  // one CTA's state in the scratch

LaPlan make_plan(const LaArgs& a, int C, size_t capacity) {
  return la_plan(a, C, kSlice, seq_sm_count(), 0.5, kStateBytes, capacity);
}

int max_d(const LaArgs& a) {
  int d = 0;
  for (int i = 0; i < a.roles; ++i) d = std::max(d, a.role[i].d);
  return d;
}
int chunk_of(int d) { return d > 64 ? Cfg<__half, 2, 2>::C : Cfg<__half, 1, 2>::C; }

template <typename T, int DB, int PARTS>
cudaError_t launch(const Maps& maps, TcArgs g, const LaPlan& p, int roles, cudaStream_t s) {
  using K = Cfg<T, DB, PARTS>;
  constexpr int smem = (int)(K::oTab + sizeof(Tables));
  static_assert(smem <= 227 * 1024 && K::oTab % 16 == 0, "shared memory");
  auto kernel = la_tc_kernel<T, DB, PARTS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned bh = (unsigned)(g.B * g.H * p.slices);
  if (p.segs > 1) {
    g.states_only = 1;
    kernel<<<dim3(bh * p.subs, roles), kThreads, smem, s>>>(maps, g);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    g.states_only = 0;
  }
  kernel<<<dim3(bh * p.segs, roles), kThreads, smem, s>>>(maps, g);
  return cudaGetLastError();
}

}  // namespace

bool la_tc_serves(const LaArgs& a) {
  if (a.dtype == PRNN_F32 || !encode_fn() || (long long)a.B * a.H * 64 * 4 >= (1LL << 31)) return false;
  for (int i = 0; i < a.roles; ++i)
    if (a.role[i].d > 128 || a.role[i].e > 128) return false;
  return true;
}

size_t la_tc_copy_bytes(const LaSeq& x, const LaArgs& a, int d) {
  if (seq_fits(x, a, d)) return 0;
  return (size_t)2 * a.T * a.B * (a.H / x.share) * ((d + 7) / 8 * 8);  // a multiple of 16
}

size_t la_tc_workspace(const LaArgs& a) {
  const LaPlan p = make_plan(a, chunk_of(max_d(a)), ~(size_t)0);
  return (size_t)a.roles * a.B * a.H * p.subs * p.slices * kStateBytes;
}

cudaError_t launch_la_tc(const LaArgs& a, void* scratch, size_t bytes, cudaStream_t s) {
  if (a.roles == 0 || a.B == 0) return cudaSuccess;
  const int d = max_d(a), C = chunk_of(d);
  const bool half = a.dtype == PRNN_F16;
  Maps maps;
  LaSeq seen[4];
  int width[4], n = 0;
  size_t used = 0;
  cudaError_t err = cudaSuccess;
  // The tensor map of x; a tensor that TMA cannot read (alignment, odd sizes, a stride of 0) is
  // copied first.
  auto index = [&](LaSeq x, int w) {
    for (int i = 0; i < n; ++i)
      if (seen[i].p == x.p && seen[i].st == x.st && seen[i].sb == x.sb && seen[i].sh == x.sh &&
          seen[i].share == x.share && width[i] == w)
        return i;
    if (n == 4) return -1;
    seen[n] = x;
    width[n] = w;
    if (const size_t copy = la_tc_copy_bytes(x, a, w)) {
      if (used + copy > bytes) return -1;
      const int heads = a.H / x.share, dp = (w + 7) / 8 * 8;
      const long long rows = (long long)a.T * a.B * heads, blocks = (rows * dp + 255) / 256;
      uint16_t* to = reinterpret_cast<uint16_t*>(static_cast<char*>(scratch) + used);
      la_copy_kernel<<<(unsigned)std::min<long long>(blocks, 16LL * seq_sm_count()), 256, 0, s>>>(
          static_cast<const uint16_t*>(x.p), x.st, x.sb, x.sh, a.B, heads, w, dp, rows, to);
      if ((err = cudaGetLastError()) != cudaSuccess) return -1;
      used += copy;
      x = LaSeq{to, (long long)a.B * heads * dp, (long long)heads * dp, dp, x.share};
      w = dp;
    }
    return encode(&maps.m[n], x, w, a.H / x.share, a.B, a.T, C, half) ? n++ : -1;
  };
  TcArgs g{};
  for (int i = 0; i < a.roles; ++i) {
    const LaRole& r = a.role[i];
    TcRole& t = g.role[i];
    t.ia = index(r.a, r.d);
    t.ib = index(r.b, r.d);
    t.ic = index(r.c, r.e);
    if (t.ia < 0 || t.ib < 0 || t.ic < 0) return err != cudaSuccess ? err : cudaErrorInvalidValue;
    t.sa = r.a.share;
    t.sb = r.b.share;
    t.sc = r.c.share;
    t.out = r.out;
    t.ot = r.ot;
    t.ob = r.ob;
    t.oh = r.oh;
    const int unit = r.out_f32 ? 4 : 8;
    const bool packs = r.e % 8 == 0 && (reinterpret_cast<uintptr_t>(r.out) & 15) == 0 &&
                (a.T == 1 || r.ot % unit == 0) && (a.B == 1 || r.ob % unit == 0) &&
                (a.H == 1 || r.oh % unit == 0);
    t.form = (packs ? 0 : kOutSingle) | (r.out_f32 ? kOutF32 : 0);
    t.d = r.d;
    t.e = r.e;
    t.x0 = r.x0;
    t.x_end = r.x_end;
    t.x_t = r.x_t;
    t.rev = r.rev;
    t.lead = r.lead;
    t.s_intra = r.s_intra;
    t.s_inter = r.s_inter;
    t.s_add = r.s_add;
  }
  for (int i = n; i < 4; ++i) maps.m[i] = maps.m[0];
  const LaPlan p = make_plan(a, C, bytes - used);
  g.T = a.T;
  g.B = a.B;
  g.H = a.H;
  g.log_decay = a.log_decay;
  g.lens = a.lens;
  g.status = seq_status_word();
  if (!g.status) return cudaErrorUnknown;
  g.segs = p.segs;
  g.cps = p.cps;
  g.subs = p.subs;
  g.cpb = p.cpb;
  g.slices = p.slices;
  g.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + used);
  bool ends = false;
  for (int i = 0; i < a.roles; ++i) ends = ends || a.role[i].x_end;
  if (half)
    return d > 64 ? launch<__half, 2, 2>(maps, g, p, a.roles, s) : launch<__half, 1, 2>(maps, g, p, a.roles, s);
  if (ends)
    return d > 64 ? launch<__nv_bfloat16, 2, 3>(maps, g, p, a.roles, s)
                  : launch<__nv_bfloat16, 1, 3>(maps, g, p, a.roles, s);
  return d > 64 ? launch<__nv_bfloat16, 2, 2>(maps, g, p, a.roles, s)
                : launch<__nv_bfloat16, 1, 2>(maps, g, p, a.roles, s);
}

}  // namespace prnn
