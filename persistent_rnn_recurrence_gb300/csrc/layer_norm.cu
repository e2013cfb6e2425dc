// layer_norm.cu -- layer norm over the last axis and its gradient.
//
// Both are bound by memory: 8 to 14 flops per element against 4 to 12 bytes.  A row is read once: the
// forward pass keeps it in registers between the sums and the output, the gradient in a ring in shared
// memory.  Measured on GB300 against the copy rate of 6.69 TB/s: forward 8192 x 5760 fp32 57 us (0.99),
// 32768 x 1152 fp32 47 (0.96), 8192 x 4096 bf16 30 (0.68: the rows, held as
// fp32 values, keep half as many bytes in flight and the loads wait); gradient 8192 x 5760 fp32 101 (0.84), 32768 x
// 1152 fp32 82 (0.83), 8192 x 4096 bf16 48 (0.62: the chain of one row's barrier and sums).  Ragged
// rows are slower for their 2- or 4-byte accesses: 8192 x 2001 bf16 28 and 40 us (0.36, 0.37).
#include <algorithm>

#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

// Sums of each of N values over the TPR threads that hold one row.  RPB rows share a block; part
// is [N][warps of the block] and may be used again after the next barrier.  TPR = 32 needs no barrier.
template <int TPR, int N, int WARPS>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*part)[WARPS]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, first = threadIdx.x / TPR * (TPR / 32);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < TPR / 32; ++w) v[i] += part[i][first + w];
    }
  }
}

template <int TPR>
constexpr int kRows = TPR >= 256 ? 1 : 256 / TPR;  // rows per block

// V parameters from an address that is a multiple of 4 bytes only when V is 1, else of 16.
template <int V>
__device__ __forceinline__ Pack<float, V> load_params(const float* p) {
  Pack<float, V> r;
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(r.v + i) = __ldg(reinterpret_cast<const float4*>(p + i));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = __ldg(p + i);
  }
  return r;
}

// Pack p of thread t in a row: columns (p * TPR + t) * V ...
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR* kRows<TPR>) layer_norm_kernel(LayerNormArgs a) {
  constexpr int WARPS = TPR * kRows<TPR> / 32;
  __shared__ float part[2][1][WARPS];
  const int t = threadIdx.x % TPR;
  const long long r = (long long)blockIdx.x * kRows<TPR> + threadIdx.x / TPR;
  const bool live = r < a.rows;
  const T* x = static_cast<const T*>(a.x) + (live ? r : 0) * a.x_stride;
  Pack<T, V> px[NV];
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    const int c = (p * TPR + t) * V;
    if (live && c < a.cols) px[p] = load_once<T, V>(x + c);
  }
  constexpr int H = V == 1 ? 1 : V / 2;  // pairs of a pack
  float2 f[NV][H];
  float2 acc = both(0.f);
#pragma unroll
  for (int p = 0; p < NV; ++p)
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const bool in = live && (p * TPR + t) * V < a.cols;
      f[p][i] = in ? pair_of<T, V>(px[p], i) : both(0.f);
      acc = add2(acc, f[p][i]);
    }
  float s[1] = {acc.x + acc.y};
  row_sum<TPR, 1, WARPS>(s, part[0]);
  // The squared distances are taken from the mean: E[x^2] - mean^2 would lose the variance of
  // rows whose mean is large.
  const float mean = s[0] / a.cols;
  acc = both(0.f);
#pragma unroll
  for (int p = 0; p < NV; ++p)
    if (live && (p * TPR + t) * V < a.cols)
#pragma unroll
      for (int i = 0; i < H; ++i) {
        f[p][i] = add2(f[p][i], both(-mean));
        acc = fma2(f[p][i], f[p][i], acc);
      }
  s[0] = V == 1 ? acc.x : acc.x + acc.y;
  row_sum<TPR, 1, WARPS>(s, part[1]);
  const float rstd = 1.f / sqrtf(s[0] / a.cols + a.eps);
  if (!live) return;
  T* y = static_cast<T*>(a.y) + r * a.y_stride;
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    const int c = (p * TPR + t) * V;
    if (c >= a.cols) continue;
    Pack<float, V> g, b;
    if (a.gamma) g = load_params<V>(a.gamma + c);
    if (a.beta) b = load_params<V>(a.beta + c);
    Pack<T, V> o;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      float2 v = mul2(f[p][i], both(rstd));
      if (a.gamma) v = mul2(v, pair_of<float, V>(g, i));
      if (a.beta) v = add2(v, pair_of<float, V>(b, i));
      set_pair<T, V>(o, i, v);
    }
    store_pack<T, V>(y + c, o);
  }
  if (t == 0) {
    if (a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
}

// Rows too long for registers: one block per row, read three times (the second and third from L2).  Columns
// are counted in 64 bits: a step past the last of nearly 2^31 does not fit 32.
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(LayerNormArgs a) {
  __shared__ float part[2][32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    T* y = static_cast<T*>(a.y) + r * a.y_stride;
    float s = 0.f;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) s += to_f32(x[c]);
    const float mean = block_sum(s, part[0]) / a.cols;
    float q = 0.f;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float d = to_f32(x[c]) - mean;
      q += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(q, part[1]) / a.cols + a.eps);
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = a.gamma ? a.gamma[c] : 1.f, b = a.beta ? a.beta[c] : 0.f;
      y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * g + b);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    __syncthreads();
  }
}

// ---- rows through shared memory -----------------------------------------------------------
//
// Persistent blocks, one per SM, of 512 threads in groups of TPR; group g of block b visits rows b*G + g,
// + grid*G, ...  Each group keeps a ring of rows (of NT tensors) in shared memory, filled by
// bulk copies a ring ahead: the memory stays busy through a row's barriers, and no registers are
// spent on prefetching.  A group takes R rows at a time, so that one chain of shuffles, barrier and
// sums serves R rows.  A row's copy covers the 16-byte lines it touches, so rows of any alignment go this
// way; what such a line holds outside the tensor (the first row's head, the last row's tail) is never
// read: those few values are copied one by one.  VEC: thread t holds packs of 16 bytes t, t + TPR,
// ...; otherwise pairs of single columns TPR apart.
constexpr int kRingThreads = 512, kRingMost = 8;

template <int NT>
struct RingArgs {
  const void* base[NT];
  long long stride[NT];   // elements
  long long bytes[NT];    // extent of the tensor
  int cols, stages;
  uint32_t pitch;         // bytes of one row's place in the ring (a multiple of 16)
  int* status;
};

// The lines of one row that lie wholly in the tensor, [from, from + bytes); the values outside them are
// copied to their places at `dst` here.
struct Lines {
  uintptr_t from;
  uint32_t skip, bytes;  // offset of `from` in the row's place, size
};
template <typename T>
__device__ __forceinline__ Lines row_lines(unsigned char* dst, uintptr_t lo, long long extent,
                                           uintptr_t s, int cols) {
  const uintptr_t hi = lo + extent, e = s + (size_t)cols * sizeof(T), at = s & ~(uintptr_t)15;
  uintptr_t from = at, to = (e + 15) & ~(uintptr_t)15;
  if (from < lo) {
    from += 16;
    for (uintptr_t p = s; p < from && p < e; p += sizeof(T))
      *reinterpret_cast<T*>(dst + (p - at)) = *reinterpret_cast<const T*>(p);
  }
  if (to > hi) {
    to -= 16;
    for (uintptr_t p = to > from ? to : from; p < e; p += sizeof(T))
      *reinterpret_cast<T*>(dst + (p - at)) = *reinterpret_cast<const T*>(p);
  }
  return {from, (uint32_t)(from - at), to > from ? (uint32_t)(to - from) : 0u};
}
__device__ __forceinline__ void copy_lines(unsigned char* dst, const Lines& l, uint64_t* bar) {
  if (l.bytes == 0) return;
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tc::smem_u32(dst + l.skip)),
      "l"(l.from), "r"(l.bytes), "r"(tc::smem_u32(bar))
      : "memory");
}

// Fill one place of the ring with row r (one thread).
template <typename T, int NT, bool VEC>
__device__ __forceinline__ void ring_fill(const RingArgs<NT>& ring, unsigned char* place,
                                          uint64_t* bar, long long r) {
  Lines l[NT];
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(ring.base[i]);
    const uintptr_t row = base + (uintptr_t)(r * ring.stride[i]) * sizeof(T);
    if constexpr (VEC)
      l[i] = {row, 0u, (uint32_t)(ring.cols * sizeof(T))};
    else
      l[i] = row_lines<T>(place + i * ring.pitch, base, ring.bytes[i], row, ring.cols);
    n += l[i].bytes;
  }
  tc::mbar_arrive_expect_tx(bar, n);
#pragma unroll
  for (int i = 0; i < NT; ++i) copy_lines(place + i * ring.pitch, l[i], bar);
}

// After a wait that ran out: report it and leave no copy in flight.  `fills`: how many this thread issued.
__device__ __noinline__ void ring_late(uint64_t* bars, int stages, int fills, int* status) {
  atomicExch(status, 1);
  bool ok = true;
  for (int i = 0; i < stages && i < fills; ++i)
    seq_wait(&bars[i], (uint32_t)((fills - 1 - i) / stages) & 1u, ok);
}

// Parameters (gamma, beta) in shared memory beside packs of V values: pack p of thread t reads its V
// floats four at a time, from places where the threads of a warp lie side by side (no bank
// conflicts).  param_place: where column c goes.
template <int V, int TPR>
__device__ __forceinline__ int param_place(int c) {
  const int pack = c / V, p = pack / TPR, t = pack % TPR, j = c % V;
  return ((p * (V / 4) + j / 4) * TPR + t) * 4 + j % 4;
}
template <int V, int TPR>
__device__ __forceinline__ Pack<float, V> param_pack(const float* s, int p, int t) {
  Pack<float, V> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    *reinterpret_cast<float4*>(r.v + 4 * i) =
        *reinterpret_cast<const float4*>(s + ((p * (V / 4) + i) * TPR + t) * 4);
  return r;
}

// Sums of N values per thread over the TPR threads of group g; part [N][warps of the group].
template <int TPR, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*part)[TPR / 32], int g, int t) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (TPR > 32) {
    if ((t & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[i][t >> 5] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(TPR) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < TPR / 32; ++w) v[i] += part[i][w];
    }
  } else {
    __syncwarp();
  }
}

// What the forward and the gradient kernels do alike: the shape of a thread's share of a row.
template <typename T, int NV, int TPR, bool VEC>
struct Share {
  static constexpr int V = 16 / sizeof(T), H = V / 2, N = NV * H, G = kRingThreads / TPR;
  static_assert(G * TPR == kRingThreads && (TPR == 32 || G <= 15), "groups");
  int t, cols;
  // columns of pair i: (col(i), col2(i))
  __device__ __forceinline__ int col(int i) const {
    return VEC ? ((i / H) * TPR + t) * V + 2 * (i % H) : 2 * i * TPR + t;
  }
  __device__ __forceinline__ int col2(int i) const { return VEC ? col(i) + 1 : col(i) + TPR; }
  // f(i, first, second...) for the pairs that lie in the row; `other` stands for a column past it
  template <typename F>
  __device__ __forceinline__ float2 single(const F* p, int i, float other) const {
    const int c = col(i), c2 = col2(i);
    return make_float2(c < cols ? to_f32(p[c]) : other, c2 < cols ? to_f32(p[c2]) : other);
  }
};

// The gradient in one pass over x and dy: dx row by row; dgamma and dbeta are summed in registers over
// the group's rows, then over the block's groups, and leave as one partial sum per block.
template <typename T, int NV, int TPR, int R, bool VEC>
__global__ void __launch_bounds__(kRingThreads, 1)
    layer_norm_grad_kernel(const __grid_constant__ LayerNormGradArgs a,
                           const __grid_constant__ RingArgs<2> ring) {
  using S = Share<T, NV, TPR, VEC>;
  constexpr int V = S::V, H = S::H, N = S::N, G = S::G;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[G][kRingMost];
  __shared__ float part[G][2][2 * R][TPR / 32];
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const S sh{t, a.cols};
  unsigned char* mine = smem + (size_t)g * ring.stages * 2 * ring.pitch;
  float* gam = reinterpret_cast<float*>(smem + (size_t)G * ring.stages * 2 * ring.pitch);
  if (t == 0) {
    for (int i = 0; i < ring.stages; ++i) tc::mbar_init(&bars[g][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const long long first = (long long)blockIdx.x * G + g, step = (long long)gridDim.x * G;
  int fills = 0;
  auto fill = [&](long long r, int s) {
    ring_fill<T, 2, VEC>(ring, mine + (size_t)s * 2 * ring.pitch, &bars[g][s], r);
    ++fills;
  };
  if (t == 0)
    for (int s = 0; s < ring.stages && first + s * step < a.rows; ++s) fill(first + s * step, s);
  for (int c = threadIdx.x; c < a.cols; c += kRingThreads)
    gam[VEC ? param_place<V, TPR>(c) : c] = a.gamma ? a.gamma[c] : 1.f;
  float2 dg[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = db[i] = both(0.f);
  float mean[R], rstd[R];
  auto stats = [&](long long r0) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool in = r0 + k * step < a.rows;
      mean[k] = in ? a.mean[r0 + k * step] : 0.f;
      rstd[k] = in ? a.rstd[r0 + k * step] : 0.f;
    }
  };
  stats(first);
  __syncthreads();
  const float inv = 1.f / a.cols;
  bool ok = true;
  int s = 0, turn = 0;
  uint32_t parity = 0;
  for (long long r = first; r < a.rows; r += R * step) {
    const T *px[R], *py[R];
    int next = s;
    uint32_t next_parity = parity;
    float m[R], rs[R], sum[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      sum[2 * k] = sum[2 * k + 1] = 0.f;
      m[k] = mean[k];
      rs[k] = rstd[k];
      px[k] = py[k] = nullptr;
      if (r + k * step < a.rows) {
        seq_wait(&bars[g][next], next_parity, ok);
        const unsigned char* at = mine + (size_t)next * 2 * ring.pitch;
        uintptr_t ox = 0, oy = 0;
        if constexpr (!VEC) {
          ox = (reinterpret_cast<uintptr_t>(a.x) + (r + k * step) * a.x_stride * sizeof(T)) & 15;
          oy = (reinterpret_cast<uintptr_t>(a.dy) + (r + k * step) * a.dy_stride * sizeof(T)) & 15;
        }
        px[k] = reinterpret_cast<const T*>(at + ox);
        py[k] = reinterpret_cast<const T*>(at + ring.pitch + oy);
        if (++next == ring.stages) {
          next = 0;
          next_parity ^= 1;
        }
      }
    }
    stats(r + R * step);
    float2 acc[R][2];
#pragma unroll
    for (int k = 0; k < R; ++k) acc[k][0] = acc[k][1] = both(0.f);
    auto first_pass = [&](int k, int i, float2 xv, float2 d, float2 gm) {
      const float2 xh = mul2(add2(xv, both(-m[k])), both(rs[k])), gg = mul2(d, gm);
      acc[k][0] = add2(acc[k][0], gg);
      acc[k][1] = fma2(gg, xh, acc[k][1]);
      dg[i] = fma2(d, xh, dg[i]);
      db[i] = add2(db[i], d);
    };
    if constexpr (VEC) {
#pragma unroll
      for (int p = 0; p < NV; ++p)
        if ((p * TPR + t) * V < a.cols) {
          const Pack<float, V> gm = param_pack<V, TPR>(gam, p, t);
#pragma unroll
          for (int k = 0; k < R; ++k)
            if (px[k]) {
              const Pack<T, V> qx = load_pack<T, V>(px[k] + (p * TPR + t) * V);
              const Pack<T, V> qy = load_pack<T, V>(py[k] + (p * TPR + t) * V);
#pragma unroll
              for (int i = 0; i < H; ++i)
                first_pass(k, p * H + i, pair_of<T, V>(qx, i), pair_of<T, V>(qy, i),
                           pair_of<float, V>(gm, i));
            }
        }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)  // past the row: x = mean and dy = 0 add nothing
        if (sh.col(i) < a.cols)
#pragma unroll
          for (int k = 0; k < R; ++k)
            if (px[k])
              first_pass(k, i, sh.single(px[k], i, m[k]), sh.single(py[k], i, 0.f),
                         sh.single(gam, i, 0.f));
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      sum[2 * k] = acc[k][0].x + acc[k][0].y;
      sum[2 * k + 1] = acc[k][1].x + acc[k][1].y;
    }
    group_sum<TPR, 2 * R>(sum, part[g][turn], g, t);
    // every thread of the group has left the rows of the turn before: their places take the rows a
    // ring ahead
    if (t == 0 && r != first) {
      int to = s;
#pragma unroll
      for (int k = R; k >= 1; --k) {
        to = to == 0 ? ring.stages - 1 : to - 1;
        const long long q = r + (ring.stages - (R - k + 1)) * step;
        if (q < a.rows) fill(q, to);
      }
    }
    if (a.dx) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (!px[k]) continue;
        const float c0 = -sum[2 * k] * inv, c1 = -sum[2 * k + 1] * inv;
        T* dx = static_cast<T*>(a.dx) + (r + k * step) * a.dx_stride;
        auto out = [&](float2 xv, float2 d, float2 gm) {
          const float2 xh = mul2(add2(xv, both(-m[k])), both(rs[k]));
          return mul2(both(rs[k]), fma2(xh, both(c1), fma2(d, gm, both(c0))));
        };
        if constexpr (VEC) {
#pragma unroll
          for (int p = 0; p < NV; ++p)
            if ((p * TPR + t) * V < a.cols) {
              const Pack<float, V> gm = param_pack<V, TPR>(gam, p, t);
              const Pack<T, V> qx = load_pack<T, V>(px[k] + (p * TPR + t) * V);
              const Pack<T, V> qy = load_pack<T, V>(py[k] + (p * TPR + t) * V);
              Pack<T, V> o;
#pragma unroll
              for (int i = 0; i < H; ++i)
                set_pair<T, V>(o, i, out(pair_of<T, V>(qx, i), pair_of<T, V>(qy, i),
                                         pair_of<float, V>(gm, i)));
              store_pack<T, V>(dx + (p * TPR + t) * V, o);
            }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (sh.col(i) < a.cols) {
              const float2 v = out(sh.single(px[k], i, m[k]), sh.single(py[k], i, 0.f),
                                   sh.single(gam, i, 0.f));
              dx[sh.col(i)] = from_f32<T>(v.x);
              if (sh.col2(i) < a.cols) dx[sh.col2(i)] = from_f32<T>(v.y);
            }
        }
      }
    }
    turn ^= 1;
    s = next;
    parity = next_parity;
  }
  if (!ok) ring_late(bars[g], ring.stages, t == 0 ? fills : 0, ring.status);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!a.partial) return;
  // partial: [2][grid][cols], the groups' sums added in order
  float* fold = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float* to = a.partial + ((size_t)w * gridDim.x + blockIdx.x) * a.cols;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 v = w ? db[i] : dg[i];
      if (sh.col(i) < a.cols) fold[(size_t)g * a.cols + sh.col(i)] = v.x;
      if (sh.col2(i) < a.cols) fold[(size_t)g * a.cols + sh.col2(i)] = v.y;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kRingThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < G; ++k) v += fold[(size_t)k * a.cols + c];
      to[c] = v;
    }
  }
}

// The forward pass of many rows that 16-byte accesses do not fit: a row's values stay in registers between the two sums and
// the output.
template <typename T, int NV, int TPR, int R>
__global__ void __launch_bounds__(kRingThreads, 1)
    layer_norm_ring_kernel(const __grid_constant__ LayerNormArgs a,
                           const __grid_constant__ RingArgs<1> ring) {
  using S = Share<T, NV, TPR, false>;
  constexpr int V = S::V, N = S::N, G = S::G;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[G][kRingMost];
  __shared__ float part[G][2][R][TPR / 32];
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const S sh{t, a.cols};
  unsigned char* mine = smem + (size_t)g * ring.stages * ring.pitch;
  float* gam = reinterpret_cast<float*>(smem + (size_t)G * ring.stages * ring.pitch);
  float* bet = gam + NV * TPR * V;
  if (t == 0) {
    for (int i = 0; i < ring.stages; ++i) tc::mbar_init(&bars[g][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const long long first = (long long)blockIdx.x * G + g, step = (long long)gridDim.x * G;
  int fills = 0;
  auto fill = [&](long long r, int s) {
    ring_fill<T, 1, false>(ring, mine + (size_t)s * ring.pitch, &bars[g][s], r);
    ++fills;
  };
  if (t == 0)
    for (int s = 0; s < ring.stages && first + s * step < a.rows; ++s) fill(first + s * step, s);
  for (int c = threadIdx.x; c < a.cols; c += kRingThreads) {
    gam[c] = a.gamma ? a.gamma[c] : 1.f;
    bet[c] = a.beta ? a.beta[c] : 0.f;
  }
  __syncthreads();
  const float inv = 1.f / a.cols;
  bool ok = true;
  int s = 0;
  uint32_t parity = 0;
  for (long long r = first; r < a.rows; r += R * step) {
    int next = s;
    uint32_t next_parity = parity;
    bool in[R];
    float2 f[R][N];
    float sum[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      in[k] = r + k * step < a.rows;
      float2 acc = both(0.f);
      if (in[k]) {
        seq_wait(&bars[g][next], next_parity, ok);
        const T* px = reinterpret_cast<const T*>(
            mine + (size_t)next * ring.pitch +
            ((reinterpret_cast<uintptr_t>(a.x) + (r + k * step) * a.x_stride * sizeof(T)) & 15));
        if (++next == ring.stages) {
          next = 0;
          next_parity ^= 1;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (sh.col(i) < a.cols) {
            f[k][i] = sh.single(px, i, 0.f);
            acc = add2(acc, f[k][i]);
          }
      }
      sum[k] = acc.x + acc.y;
    }
    group_sum<TPR, R>(sum, part[g][0], g, t);
    // the rows are in registers: their places take the rows a ring ahead
    if (t == 0) {
      int to = s;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const long long q = r + (ring.stages + k) * step;
        if (q < a.rows) fill(q, to);
        if (++to == ring.stages) to = 0;
      }
    }
    float mean[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mean[k] = sum[k] * inv;
      float2 acc = both(0.f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (sh.col(i) < a.cols) {
          f[k][i] = add2(f[k][i], both(-mean[k]));
          if (sh.col2(i) >= a.cols) f[k][i].y = 0.f;
          acc = fma2(f[k][i], f[k][i], acc);
        }
      sum[k] = acc.x + acc.y;
    }
    group_sum<TPR, R>(sum, part[g][1], g, t);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (!in[k]) continue;
      const float rstd = 1.f / sqrtf(sum[k] * inv + a.eps);
      T* y = static_cast<T*>(a.y) + (r + k * step) * a.y_stride;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (sh.col(i) < a.cols) {
          const float2 v = fma2(mul2(f[k][i], both(rstd)), sh.single(gam, i, 0.f),
                                sh.single(bet, i, 0.f));
          y[sh.col(i)] = from_f32<T>(v.x);
          if (sh.col2(i) < a.cols) y[sh.col2(i)] = from_f32<T>(v.y);
        }
      if (t == 0) {
        if (a.mean) a.mean[r + k * step] = mean[k];
        if (a.rstd) a.rstd[r + k * step] = rstd;
      }
    }
    s = next;
    parity = next_parity;
  }
  if (!ok) ring_late(bars[g], ring.stages, t == 0 ? fills : 0, ring.status);
}

// dx of rows too long for registers, and their sums (partial: [2][splits][cols]).
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_dx_long_kernel(LayerNormGradArgs a) {
  __shared__ float part[2][32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s = 0.f, q = 0.f;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(dy[c]) * (a.gamma ? a.gamma[c] : 1.f);
      s += g;
      q += g * ((to_f32(x[c]) - mean) * rstd);
    }
    s = block_sum(s, part[0]) / a.cols;
    q = block_sum(q, part[1]) / a.cols;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(dy[c]) * (a.gamma ? a.gamma[c] : 1.f);
      dx[c] = from_f32<T>(rstd * (g - s - (to_f32(x[c]) - mean) * rstd * q));
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void layer_norm_dw_long_kernel(LayerNormGradArgs a, int splits) {
  __shared__ float pg[32][33], pb[32][33];
  const int tx = threadIdx.x, ty = threadIdx.y;
  const long long c = blockIdx.x * 32LL + tx;
  const long long share = (a.rows + splits - 1) / splits;
  const long long lo = blockIdx.y * share, hi = lo + share < a.rows ? lo + share : a.rows;
  float g = 0.f, b = 0.f;
  if (c < a.cols)
    for (long long r = lo + ty; r < hi; r += 32) {
      const float d = to_f32(static_cast<const T*>(a.dy)[r * a.dy_stride + c]);
      g += d * (to_f32(static_cast<const T*>(a.x)[r * a.x_stride + c]) - a.mean[r]) * a.rstd[r];
      b += d;
    }
  pg[ty][tx] = g;
  pb[ty][tx] = b;
  __syncthreads();
  if (ty == 0 && c < a.cols) {
    g = b = 0.f;
    for (int i = 0; i < 32; ++i) {
      g += pg[i][tx];
      b += pb[i][tx];
    }
    a.partial[(size_t)blockIdx.y * a.cols + c] = g;
    a.partial[(size_t)(splits + blockIdx.y) * a.cols + c] = b;
  }
}

// Joins the partial sums [2][splits][cols]: 32 columns per block, its 8 rows of threads share the splits;
// a fixed order of additions.
__global__ void __launch_bounds__(256) layer_norm_dw_join_kernel(const float* partial, int splits,
                                                                 int cols, float* dgamma,
                                                                 float* dbeta) {
  __shared__ float sum[8][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const long long c = blockIdx.x * 32LL + tx;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const float* p = partial + (size_t)blockIdx.y * splits * cols;
  float v = 0.f;
  if (c < cols)
#pragma unroll 8
    for (int i = ty; i < splits; i += 8) v += p[(size_t)i * cols + c];
  sum[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += sum[k][tx];
    out[c] = v;
  }
}

constexpr int kGradBlocks = 160;  // at most: one per SM

bool vec_ok(const void* p, long long stride, size_t esz) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * (long long)esz)) & 15) == 0;
}

template <typename T, int V, int NV, int TPR>
bool run(const LayerNormArgs& a, cudaStream_t s) {
  const long long blocks = (a.rows + kRows<TPR> - 1) / kRows<TPR>;
  layer_norm_kernel<T, V, NV, TPR><<<(unsigned)blocks, TPR * kRows<TPR>, 0, s>>>(a);
  return true;
}

// Packs per thread and threads per row.  With fewer than two rows an SM there is room for all rows at
// once, and many threads a row are fastest (4 x 1792 fp32 2.4 us against 3.7 with the plans below, 300 x
// 1152 2.6 against 4.4; 600 rows of 512 bf16 values take 2.5 either way, 1200 of them 3.9 against
// 2.5).  Else the fewest threads that hold the row at up to 40 values each: a warp per row needs no
// barrier (32768 x 1152 fp32: 47 us against 54 with 128 threads, 70 with 256), and more values cost the
// occupancy that hides the loads (8192 x 4096 bf16: 30 us at 32 values, 39 at 64, 47 at 128).
template <typename T, int V>
bool pick(const LayerNormArgs& a, cudaStream_t s) {
  const int packs = (a.cols + V - 1) / V;
  if (packs <= 32) return run<T, V, 1, 32>(a, s);
  if (a.rows < 2LL * seq_sm_count()) {
    if (packs <= 256) return run<T, V, 1, 256>(a, s);
    if (packs <= 512) return run<T, V, 2, 256>(a, s);
    if (packs <= 1024) return run<T, V, 4, 256>(a, s);
    if (packs <= 2048) return run<T, V, 4, 512>(a, s);
    if (packs <= 4096) return run<T, V, 4, 1024>(a, s);
  }
  if constexpr (V > 1) {
    if (packs <= 64) return run<T, V, 2, 32>(a, s);
    if (packs <= 128) return run<T, V, 4, 32>(a, s);
  }
  if constexpr (V == 8) {
    if (packs <= 160) return run<T, V, 5, 32>(a, s);
    if (packs <= 256) return run<T, V, 4, 64>(a, s);
    if (packs <= 512) return run<T, V, 4, 128>(a, s);
    if (packs <= 1024) return run<T, V, 4, 256>(a, s);
    if (packs <= 2048) return run<T, V, 4, 512>(a, s);
    if (packs <= 4096) return run<T, V, 4, 1024>(a, s);
  } else if constexpr (V == 4) {
    if (packs <= 192) return run<T, V, 6, 32>(a, s);
    if (packs <= 320) return run<T, V, 10, 32>(a, s);
    if (packs <= 512) return run<T, V, 8, 64>(a, s);
    if (packs <= 1024) return run<T, V, 8, 128>(a, s);
    if (packs <= 2048) return run<T, V, 8, 256>(a, s);
    if (packs <= 4096) return run<T, V, 4, 1024>(a, s);
  } else {  // the rest goes through shared memory
    if (packs <= 8192) return run<T, V, 16, 512>(a, s);
  }
  return false;
}

// ---- plans of the ring kernels ------------------------------------------------------------
// NV packs of 16 bytes per thread, TPR threads per row, R rows a turn.  The gradient keeps two
// accumulators a column, so a thread takes at most 24 columns; R = 2 where the ring holds at least
// four rows a group.
template <typename T, int NV, int TPR, int NT>
bool make_ring(RingArgs<NT>& ring, bool vec, size_t params, int rows_a_turn, size_t* smem) {
  constexpr int G = kRingThreads / TPR;
  if ((size_t)ring.cols * sizeof(T) > (size_t)16 * NV * TPR) return false;
  ring.pitch = (uint32_t)(((size_t)ring.cols * sizeof(T) + 15) / 16 * 16 + (vec ? 0 : 16));
  const size_t stage = (size_t)G * NT * ring.pitch, beside = params * sizeof(float) * NV * TPR * (16 / sizeof(T));
  ring.stages = (int)std::min<size_t>(kRingMost, (220 * 1024 - beside) / stage);
  ring.status = seq_status_word();
  *smem = ring.stages * stage + beside;
  return ring.status && ring.stages >= 2 * rows_a_turn;
}

template <typename T, int NV, int TPR, int R>
cudaError_t run_grad(const LayerNormGradArgs& a, bool vec, int sms, int* blocks, cudaStream_t s) {
  constexpr int G = kRingThreads / TPR;
  RingArgs<2> ring{};
  const long long n = (long long)sizeof(T);
  ring.base[0] = a.x;
  ring.base[1] = a.dy;
  ring.stride[0] = a.x_stride;
  ring.stride[1] = a.dy_stride;
  ring.bytes[0] = ((a.rows - 1) * a.x_stride + a.cols) * n;
  ring.bytes[1] = ((a.rows - 1) * a.dy_stride + a.cols) * n;
  ring.cols = a.cols;
  size_t smem = 0;
  if (!make_ring<T, NV, TPR, 2>(ring, vec, 1, R, &smem)) return cudaErrorInvalidConfiguration;
  *blocks = (int)std::min<long long>((a.rows + G - 1) / G, std::min(sms, kGradBlocks));
  auto kernel = vec ? layer_norm_grad_kernel<T, NV, TPR, R, true>
                    : layer_norm_grad_kernel<T, NV, TPR, R, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<*blocks, kRingThreads, smem, s>>>(a, ring);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_grad(const LayerNormGradArgs& a, bool vec, int sms, int* blocks, cudaStream_t s) {
  const int packs = (int)((a.cols * sizeof(T) + 15) / 16);
  if (packs <= 32) return run_grad<T, 1, 32, 2>(a, vec, sms, blocks, s);
  if (packs <= 64) return run_grad<T, 2, 32, 2>(a, vec, sms, blocks, s);
  if (packs <= 128) return run_grad<T, 1, 128, 2>(a, vec, sms, blocks, s);
  if (packs <= 256) return run_grad<T, 2, 128, 2>(a, vec, sms, blocks, s);
  // four groups a block where their ring of fp32 rows still fits twice: 32768 x 1152 82 us against 96
  if (packs <= 512 && sizeof(T) == 4) return run_grad<T, 4, 128, 1>(a, vec, sms, blocks, s);
  if (packs <= 512) return run_grad<T, 2, 256, 2>(a, vec, sms, blocks, s);
  if (packs <= 1024) return run_grad<T, 2, 512, 2>(a, vec, sms, blocks, s);
  if constexpr (sizeof(T) == 4)
    return packs <= 1536 ? run_grad<T, 6, 256, 1>(a, vec, sms, blocks, s)
                         : run_grad<T, 4, 512, 1>(a, vec, sms, blocks, s);
  else
    return run_grad<T, 3, 512, 1>(a, vec, sms, blocks, s);
}

template <typename T, int NV, int TPR, int R>
cudaError_t run_ring(const LayerNormArgs& a, int sms, cudaStream_t s) {
  constexpr int G = kRingThreads / TPR;
  RingArgs<1> ring{};
  ring.base[0] = a.x;
  ring.stride[0] = a.x_stride;
  ring.bytes[0] = ((a.rows - 1) * a.x_stride + a.cols) * (long long)sizeof(T);
  ring.cols = a.cols;
  size_t smem = 0;
  if (!make_ring<T, NV, TPR, 1>(ring, false, 2, R, &smem)) return cudaErrorInvalidConfiguration;
  const int blocks = (int)std::min<long long>((a.rows + G - 1) / G, sms);
  auto kernel = layer_norm_ring_kernel<T, NV, TPR, R>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, kRingThreads, smem, s>>>(a, ring);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_ring(const LayerNormArgs& a, int sms, cudaStream_t s) {
  const int packs = (int)((a.cols * sizeof(T) + 15) / 16);
  if (packs <= 32) return run_ring<T, 1, 32, 2>(a, sms, s);
  if (packs <= 64) return run_ring<T, 2, 32, 2>(a, sms, s);
  if (packs <= 128) return run_ring<T, 1, 128, 2>(a, sms, s);
  if (packs <= 256) return run_ring<T, 2, 128, 2>(a, sms, s);
  if (packs <= 512) return run_ring<T, 2, 256, 2>(a, sms, s);
  if (packs <= 1024) return run_ring<T, 2, 512, 2>(a, sms, s);
  if constexpr (sizeof(T) == 4)
    return run_ring<T, 4, 512, 2>(a, sms, s);
  else
    return run_ring<T, 3, 512, 1>(a, sms, s);
}
// The longest rows they take, in 16-byte packs.
constexpr int ring_max_packs(size_t esz) { return esz == 4 ? 2048 : 1536; }

}  // namespace

// Blocks of the gradient: at most one per SM (two dies of at most 80 SMs).
int layer_norm_splits(long long rows, int) {
  return (int)(rows < 1 ? 1 : (rows > kGradBlocks ? kGradBlocks : rows));
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const size_t esz = a.dtype == PRNN_F32 ? 4 : 2;
  const bool vec = a.rows < (1LL << 31) && a.cols % (16 / esz) == 0 &&
                   vec_ok(a.x, a.rows > 1 ? a.x_stride : 0, esz) &&
                   vec_ok(a.y, a.rows > 1 ? a.y_stride : 0, esz) && vec_ok(a.gamma, 0, 4) &&
                   vec_ok(a.beta, 0, 4);
  bool done = false;
  const long long packs = ((long long)a.cols * (long long)esz + 15) / 16;
  // Through shared memory where 16-byte accesses do not fit the rows and there are two rows or more an SM:
  // 8192 x 2001 bf16 28 us against 64, 20000 x 301 fp16 16 against 24, but 300 x 2001 bf16 5.8 against
  // 3.2.  Rows that they fit are faster from registers: 8192 x 5760 fp32 57 against 71.
  if (!vec && packs <= ring_max_packs(esz) && a.rows >= 2LL * seq_sm_count()) {
    cudaError_t e = cudaSuccess;
    PRNN_BY_DTYPE(a.dtype, T, (e = pick_ring<T>(a, seq_sm_count(), s)));
    return e;
  }
  if (vec) {
    PRNN_BY_DTYPE(a.dtype, T, (done = pick<T, 16 / sizeof(T)>(a, s)));
  } else if (a.rows < (1LL << 31)) {
    PRNN_BY_DTYPE(a.dtype, T, (done = pick<T, 1>(a, s)));
  }
  if (!done) {
    const int blocks = (int)(a.rows < 65536 ? a.rows : 65536);
    PRNN_BY_DTYPE(a.dtype, T, (layer_norm_long_kernel<T><<<blocks, 1024, 0, s>>>(a)));
  }
  return cudaGetLastError();
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& args, cudaStream_t s) {
  LayerNormGradArgs a = args;
  const bool sums = a.dgamma || a.dbeta;
  if (!sums) a.partial = nullptr;
  if (!sums && !a.dx) return cudaSuccess;
  const size_t esz = a.dtype == PRNN_F32 ? 4 : 2;
  const bool one = a.rows == 1;
  const bool vec = a.cols % (16 / esz) == 0 && vec_ok(a.x, one ? 0 : a.x_stride, esz) &&
                   vec_ok(a.dy, one ? 0 : a.dy_stride, esz) &&
                   vec_ok(a.dx, one || !a.dx ? 0 : a.dx_stride, esz);
  int splits = layer_norm_splits(a.rows, a.cols);
  cudaError_t e = cudaSuccess;
  const long long packs = ((long long)a.cols * (long long)esz + 15) / 16;
  if (packs <= ring_max_packs(esz)) {
    PRNN_BY_DTYPE(a.dtype, T, (e = pick_grad<T>(a, vec, seq_sm_count(), &splits, s)));
    if (e != cudaSuccess) return e;
  } else {
    const int blocks = (int)(a.rows < 65536 ? a.rows : 65536);
    if (a.dx) {
      PRNN_BY_DTYPE(a.dtype, T, (layer_norm_dx_long_kernel<T><<<blocks, 1024, 0, s>>>(a)));
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (sums) {
      const long long want = (a.rows + 63) / 64;
      if (want < splits) splits = (int)want;
      const dim3 grid((unsigned)((a.cols + 31LL) / 32), splits);
      PRNN_BY_DTYPE(a.dtype, T,
                    (layer_norm_dw_long_kernel<T><<<grid, dim3(32, 32), 0, s>>>(a, splits)));
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  }
  if (!sums) return cudaSuccess;
  // launched as the gradient kernel's programmatic dependent: its launch overlaps that kernel's end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.cols + 31LL) / 32), 2);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_norm_dw_join_kernel, (const float*)a.partial, splits, a.cols,
                            a.dgamma, a.dbeta);
}

}  // namespace prnn
