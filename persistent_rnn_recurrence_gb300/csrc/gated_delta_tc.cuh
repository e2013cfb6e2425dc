// gated_delta_tc.cuh -- what the gated delta rule's tensor-core kernels share.
//
// A chunk of C tokens entered with the state S0, G the running sum of its log-decays, D_ij = exp(G_i - G_j) for
// j <= i:
//   M = strict_lower((K K^T) o D),   Tt = (I + M diag(beta))^-1,   W = Tt diag(e^G) K,
//   E = Tt V - W S0,   U = beta E,   o = scale (e^G Q S0 + ((Q K^T) o D) U),   S <- e^G_C S0 + (e^(G_C - G) K)^T U;
// and backwards, R the loss's gradient by the state that leaves it, dO times scale:
//   X = ((Q K^T) o D)^T dO + e^(G_C - G) K R,   R <- e^G_C R + (e^G Q)^T dO - W^T (beta X),   dV = Tt^T (beta X),
//   dbeta_i = e_i . du_i,  du_i = dv_i / beta_i = x_i - sum_{j > i} M_ji dv_j,
//   Y = strict_lower((dV U^T) o D), Z = (dO U^T) o D:
//   dQ = e^G dO S0^T + Z K,   dK = e^(G_C - G) U R^T + Z^T Q - (Y + Y^T) K - e^G dV S0^T,
//   dlog_decay_t = sum_{i >= t} (q_i . dq_i - v_i . dv_i) + <S_C, R>.
// All but the two lines with S0 and R on both sides go chunk by chunk side by side; those are walked by one kernel in
// two roles.
//
// Every operand is a sum of bf16 parts: the data exactly (bf16 one part, fp16 two, fp32 three of 8 bits each), what is
// computed in between three (24 bits), two where it feeds 16-bit outputs only; products of parts below 2^-24 of the
// whole are left out, all sums are fp32.  bf16 has fp32's range, so nothing is scaled to fit.  Log-decays are
// summed in 64 bits and kept as two fp32 values, so that differences of distant sums keep their bits; one below
// -1000 counts as -1000 (exp is 0 from -104), which keeps those differences finite.
//
// Blocks of the side-by-side kernels work in step: place operands, multiply, read.  Each runs through its code once a
// chunk, so code that is fetched costs as much as code that works: what many steps share is a function of its own
// (noinline), and data that 16-byte loads do not fit is copied beforehand (the gradients kernel of 210 KB of code took
// 550 us for T = 2048, 4 sequences of 16 heads of 128 x 128 bf16).
#pragma once

#include "gated_delta.h"
#include "seq_tc.cuh"

namespace prnn {
namespace gd {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int C = 128, kP = 3;                        // tokens per chunk; parts of computed values
constexpr uint32_t kTile = 16384;                     // [128][64] bf16, 128-byte swizzled
template <typename T>
constexpr int kData = std::is_same<T, float>::value ? 3 : (std::is_same<T, __half>::value ? 2 : 1);

// Per chunk and head, fp32 [128] each: sums G of log-decays (to the base 2) as a value and the rest of it, their exponentials, those to
// the chunk's end, betas; and the decays from each token to the last of its block of 16.
struct Gates {
  float2 sum[C];
  float up[C], down[C], beta[C], to_last[C];
};

struct Args {
  GdArgs a;
  int chunks, bh0, nbh;        // chunks of T; the heads of this launch: bh0 ... bh0 + nbh
  int dkt, dvt;                // tiles of 64 columns
  int* status;
  // scratch per (head, chunk): W and K as operand tiles [dkt][parts][128][64]; fp32 matrices in quads of
  // columns, [cols / 4][rows][4]: E and X [128][64 dvt], states (a slot more per head) and their gradients
  // [64 dkt][64 dvt], Tt [128][128], Z0 = (e^G Q)^T dO
  unsigned char *wimg, *kimg;
  Gates* gates;
  float *E, *S, *inv, *X, *Z0, *R;
};

__device__ __forceinline__ int length_of(const GdArgs& a, int b) {
  int len = a.T;
  if (a.lens) {
    len = a.lens[b];
    len = len < 0 ? 0 : (len > a.T ? a.T : len);
  }
  return len;
}
struct Place {  // of one block: a head's chunk
  int bh, b, h, hq, c, n, len;
  size_t at, slot;  // index of the chunk's scratch, of its state
  long long t0;
};
__device__ __forceinline__ Place place_of(const Args& g, int index) {
  Place p;
  const int local = index / g.chunks;
  p.c = index % g.chunks;
  p.bh = g.bh0 + local;
  p.b = p.bh / g.a.H;
  p.h = p.bh % g.a.H;
  p.hq = p.h / g.a.q.share;
  p.len = length_of(g.a, p.b);
  p.t0 = (long long)p.c * C;
  const long long left = p.len - p.t0;
  p.n = left < 0 ? 0 : (left > C ? C : (int)left);
  p.at = (size_t)local * g.chunks + p.c;
  p.slot = (size_t)local * (g.chunks + 1) + p.c;
  return p;
}
// The next of a block's chunks, from `index` in steps of the grid, that has tokens; n = 0 where there is none.
__device__ __forceinline__ Place next_place(const Args& g, int& index) {
  Place p{};
  for (; index < g.nbh * g.chunks; index += gridDim.x) {
    p = place_of(g, index);
    if (p.n > 0) return p;
  }
  p.n = 0;
  return p;
}
template <typename T>
__device__ __forceinline__ const T* rows_of(const LaSeq& x, long long t0, int b, int head) {
  return static_cast<const T*>(x.p) + t0 * x.st + b * x.sb + head * x.sh;
}

// 2^x, to about 2^-22 of itself, results below 2^-126 to 0.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(G_i - G_j) of sums to the base 2.
__device__ __forceinline__ float decay_between(float2 i, float2 j) { return exp2_of((i.x - j.x) + (i.y - j.y)); }
__device__ __forceinline__ float decay_between(const Gates& g, int i, int j) { return decay_between(g.sum[i], g.sum[j]); }
__device__ __forceinline__ float at_of16(const float2 (&v)[8], int i) { return i & 1 ? v[i / 2].y : v[i / 2].x; }
__device__ __forceinline__ void set16(float2 (&v)[8], int i, float f) {
  if (i & 1) v[i / 2].y = f;
  else v[i / 2].x = f;
}
// Columns c0 ... c0 + 15 of row `row`, both within one chunk, times D_ij: zeros where j > row (or j == row if STRICT).
// A warp's rows are 32 w ...  Blocks of columns before those take one exponential a row, since a way over the block's last
// token has two factors that are decays themselves; the diagonal ones one for each value.
template <bool STRICT>
__device__ __forceinline__ void decayed(float2 (&v)[8], int row, int c0, const Gates& g) {
  const int w = row >> 5, cw = c0 >> 5;
  if (cw > w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = both(0.f);
  } else if (cw < w) {
    const float2 f = both(decay_between(g, row, c0 + 15));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 t = *reinterpret_cast<const float4*>(g.to_last + c0 + 2 * i);
      v[i] = mul2(v[i], mul2(f, make_float2(t.x, t.y)));
      v[i + 1] = mul2(v[i + 1], mul2(f, make_float2(t.z, t.w)));
    }
  } else {
    const float2 mine = g.sum[row];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float f = at_of16(v, i) * decay_between(mine, g.sum[c0 + i]);
      set16(v, i, (STRICT ? c0 + i < row : c0 + i <= row) ? f : 0.f);
    }
  }
}

// 8 values of row r, columns 8 chunk ..., as P parts into tiles `stride` bytes apart.
template <int P>
__device__ __forceinline__ void put8(unsigned char* tile, uint32_t stride, int r, int chunk, float2 (&v)[4]) {
  const uint32_t at = (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4));
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint4 u;
    u.x = take<bf16>(v[0]);
    u.y = take<bf16>(v[1]);
    u.z = take<bf16>(v[2]);
    u.w = take<bf16>(v[3]);
    *reinterpret_cast<uint4*>(tile + p * stride + at) = u;
  }
}

// 8 values from a multiple of 16 bytes.
template <typename T>
__device__ __forceinline__ Pack<T, 8> get8(const T* p) {
  Pack<T, 8> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(&r)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ Pack<T, 8> zeros8() {
  Pack<T, 8> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(&r)[i] = make_uint4(0, 0, 0, 0);
  return r;
}
template <typename T>
__device__ __forceinline__ void pairs_of(const Pack<T, 8>& r, float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair_of<T, 8>(r, i);
}

// ROWS rows of a data tensor (from its row of the chunk's token 0), TILES tiles of 64 columns at most, requested by
// NT threads at once and later placed as P parts: rows past n and columns past d are zeros.
template <typename T, int ROWS, int TILES, int NT>
struct DataRows {
  static constexpr int N = (ROWS * 8 * TILES + NT - 1) / NT;
  Pack<T, 8> raw[N];
  int shift;  // neighbouring threads take a row's pieces of 8 columns
  __device__ __forceinline__ void fetch(const T* x, long long st, int r0, int n, int c0, int d, int tiles) {
    shift = TILES == 2 && tiles == 2 ? 4 : 3;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = i * NT + threadIdx.x, r = r0 + (u >> shift), c = c0 + (u & ((1 << shift) - 1)) * 8;
      raw[i] = (u >> shift) < ROWS && r < n && c < d ? get8<T>(x + r * st + c) : zeros8<T>();
    }
  }
  // Tiles `tile` bytes apart, parts `part` apart; each row times scale[row] where that is given.
  template <int P>
  __device__ __forceinline__ void place(unsigned char* to, uint32_t part, uint32_t tile, const float* scale = nullptr) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = i * NT + threadIdx.x, r = u >> shift, piece = u & ((1 << shift) - 1);
      if (r >= ROWS) continue;
      float2 v[4];
      pairs_of<T>(raw[i], v);
      if (scale)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], both(scale[r]));
      put8<P>(to + (piece >> 3) * tile, part, r, piece & 7, v);
    }
  }
};
// The same for an fp32 matrix of R <= ROWS rows in quads of columns; a row per lane.
template <int ROWS, int TILES, int NT>
struct QuadRows {
  static constexpr int N = (ROWS * 8 * TILES + NT - 1) / NT;
  float4 a[N], b[N];
  __device__ __forceinline__ void fetch(const float* m, int R, int rows, int tiles) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = i * NT + threadIdx.x, r = u % ROWS, piece = u / ROWS;
      if (r < rows && piece < 8 * tiles) {
        const float4* q = reinterpret_cast<const float4*>(m) + ((size_t)(2 * piece) * R + r);
        a[i] = q[0];
        b[i] = q[R];
      }
    }
  }
  template <int P>
  __device__ __forceinline__ void place(unsigned char* to, uint32_t part, uint32_t tile, int rows, int tiles,
                                        const float* scale = nullptr) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = i * NT + threadIdx.x, r = u % ROWS, piece = u / ROWS;
      if (r >= rows || piece >= 8 * tiles) continue;
      float2 v[4] = {make_float2(a[i].x, a[i].y), make_float2(a[i].z, a[i].w), make_float2(b[i].x, b[i].y),
                     make_float2(b[i].z, b[i].w)};
      if (scale)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], both(scale[r]));
      put8<P>(to + (piece >> 3) * tile, part, r, piece & 7, v);
    }
  }
};

// The whole of that, for operands that are not worth their registers earlier.
template <int P, int NT>
__device__ __noinline__ void load_quads(unsigned char* to, uint32_t part, const float* m, int rows, int tiles,
                                        const float* scale) {
  QuadRows<C, 2, NT> q;
  q.fetch(m, rows, rows, tiles);
  q.template place<P>(to, part, kTile, rows, tiles, scale);
}

// Brings `bytes` bytes from a multiple of 16 into L2.
__device__ __forceinline__ void ask_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// An operand: descriptor of its first part, bytes from one part to the next, and of its steps of 16 along K.
struct Operand {
  uint64_t desc;
  uint32_t part, tile;  // units of 16 bytes; tile 0: MN-major, K along the rows
  __device__ __forceinline__ uint64_t at(int p, int k) const {
    return desc + p * part + (tile ? (k >> 2) * tile + (k & 3) * 2 : k * 128);
  }
};
__device__ __forceinline__ Operand k_major(uint32_t addr, uint32_t part, uint32_t tile) {
  return {sw128_kmajor_desc(addr), part >> 4, tile >> 4};
}
__device__ __forceinline__ Operand mn_major(uint32_t addr, uint32_t part, uint32_t tile) {
  return {mn_desc(addr, tile), part >> 4, 0};
}
// D (+)= A B over `steps` steps of 16: every pair of parts whose places add up to MOST at most, small ones first.
static __device__ __noinline__ void product_of(int pa, int pb, int most, uint32_t d, Operand a, Operand b, int steps,
                                               uint32_t id, uint32_t acc) {
  const uint32_t step_a = a.tile ? 2 : 128, step_b = b.tile ? 2 : 128, tile_a = a.tile ? a.tile : 512,
                 tile_b = b.tile ? b.tile : 512;
#pragma unroll 1
  for (int s = min(pa + pb - 2, most); s >= 0; --s)
#pragma unroll 1
    for (int p = max(0, s - pb + 1); p < min(pa, s + 1); ++p) {
      uint64_t da = a.desc + p * a.part, db = b.desc + (s - p) * b.part;
#pragma unroll 1
      for (int k = 0; k < steps; k += 4, da += tile_a, db += tile_b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k + j < steps) {
            umma_f16(d, da + j * step_a, db + j * step_b, id, acc);
            acc = 1;
          }
    }
}
template <int PA, int PB, int MOST = 2>
__device__ __forceinline__ void product(uint32_t d, const Operand& a, const Operand& b, int steps, uint32_t id,
                                        bool add) {
  product_of(PA, PB, MOST, d, a, b, steps, id, add);
}
__device__ __forceinline__ uint32_t id_of(int n, bool a_mn, bool b_mn) {
  return bf16_idesc(128, n) | (a_mn ? kAMn : 0u) | (b_mn ? kBMn : 0u);
}

template <int NT>
__device__ __forceinline__ void copy_gates(Gates& to, const Gates* from) {
  for (int i = threadIdx.x; i < (int)(sizeof(Gates) / 4); i += NT)
    reinterpret_cast<float*>(&to)[i] = reinterpret_cast<const float*>(from)[i];
}

// Blocks that work in step: operands are placed by all threads, one thread issues the products, all wait for them.
struct Steps {
  uint64_t* bar;
  uint32_t turn = 0;
  bool ok = true;
  template <typename F>
  __device__ __forceinline__ void run(F&& issue) {
    to_async();
    before_sync();
    __syncthreads();
    if (threadIdx.x < 32) {
      if (elected()) {
        after_sync();
        issue();
        umma_commit(bar);
      }
      __syncwarp();
    }
  }
  // Every thread polls: a barrier behind one polling warp took longer (371 us of the gradients against 359).
  __device__ __forceinline__ void wait() {
    seq_wait(bar, turn & 1, ok);
    ++turn;
    __syncwarp();
    after_sync();
  }
};

// Set-up and end of a block that works in step: a barrier and `cols` columns of tensor memory.
__device__ __forceinline__ bool begin(uint64_t* bar, uint32_t* tmem, uint32_t cols, const unsigned char* smem,
                                      int* status) {
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it; no static shared memory precedes them
    if (threadIdx.x == 0) atomicExch(status, 1);
    return false;
  }
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < 32) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  return true;
}
__device__ __forceinline__ void finish(uint32_t tmem, uint32_t cols, bool ok, int* status) {
  if (!ok) atomicExch(status, 1);
  before_sync();
  __syncthreads();
  if (threadIdx.x < 32) {
    after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  }
}

// 16 columns of this thread's row of an accumulator.
__device__ __forceinline__ void read16(uint32_t at, float2 (&v)[8]) {
  uint32_t r[16];
  tmem_ld16(at, r);
  wait_ld();
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = pair_at(r, i);
}
// 16 columns c0 ... of row r to an fp32 matrix of R rows in quads.
__device__ __forceinline__ void store_quads(float* m, int R, int r, int c0, const float2 (&v)[8]) {
  float4* q = reinterpret_cast<float4*>(m) + ((size_t)(c0 / 4) * R + r);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[(size_t)i * R] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
}
// 16 values as P parts: row r, columns c0 ... of tiles of 64 columns, parts `stride` bytes apart.
template <int P>
__device__ __forceinline__ void put16(unsigned char* tiles, uint32_t stride, int r, int c0, const float2 (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float2 w[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
    put8<P>(tiles + (c0 >> 6) * kTile, stride, r, ((c0 & 63) >> 3) + j, w);
  }
}
// 16 values of one row at p, of which the first m, a multiple of 8, are the output's.
template <typename T>
__device__ __forceinline__ void store16(T* p, int m, const float2 (&v)[8]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / V; ++i) {
    if (i * V >= m) continue;
    Pack<T, V> o;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) set_pair<T, V>(o, j, v[i * V / 2 + j]);
    store_pack<T, V>(p + i * V, o);
  }
}

__device__ __forceinline__ void times16(float2 (&v)[8], const float* f) {  // f: 16 floats, 16-byte aligned
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 t = *reinterpret_cast<const float4*>(f + 2 * i);
    v[i] = mul2(v[i], make_float2(t.x, t.y));
    v[i + 1] = mul2(v[i + 1], make_float2(t.z, t.w));
  }
}

// `per_sm` blocks an SM where each has chunks enough to go on with the next, else one for every chunk.
inline unsigned grid_of(const Args& g, int per_sm) {
  const long long n = (long long)g.nbh * g.chunks, at_once = (long long)per_sm * seq_sm_count();
  return (unsigned)(n < 4 * at_once ? n : at_once);
}

cudaError_t launch_prepare(const Args& g, bool keep_inverse, cudaStream_t s);
cudaError_t launch_chain(const Args& g, bool reverse, cudaStream_t s);
cudaError_t launch_outputs(const Args& g, cudaStream_t s);
cudaError_t launch_before_reverse(const Args& g, cudaStream_t s);
cudaError_t launch_gradients(const Args& g, cudaStream_t s);

}  // namespace gd
}  // namespace prnn
