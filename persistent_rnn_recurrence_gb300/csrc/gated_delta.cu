// gated_delta.cu -- the gated delta rule on CUDA cores, token by token, for any sizes, strides and types:
//   S' = a S_{t-1},  e_t = v_t - S'^T k_t,  S_t = S' + k_t (beta_t e_t)^T,  o_t = scale S_t^T q_t,
// and its gradient, with R the loss's gradient by S_t:
//   R += scale q_t do_t^T,  du = R^T k_t,  dv_t = beta_t du,  dbeta_t = e_t . du,
//   dk_t = R (beta_t e_t) - S' dv_t,  dq_t = scale S_t do_t,  R <- a (R - k_t dv_t^T).
//
// Columns of S and of R never meet within the recurrences of e and du, and rows never meet once e and du are
// known.  So four walks: e forwards and du backwards over columns, dq and half of dk forwards and the other half
// backwards over rows.  A lane of 8 holds every 8th quad of a column (or row), whose dot products take three
// shuffles; the vectors of a block of tokens are staged in shared memory while the block before is worked on.
// The decays' gradient <S', R'> is taken apart per block of kGdBlock tokens: moving the decay of one token scales all
// that comes after it, so dlog_decay_t = sum over i >= t of the block of (q_i . dq_i - v_i . dv_i) + <S, R> at its end.
//
// Bound by the chain of a token in the first two walks (dot product, three shuffles, update) and the blocks' staging where
// warps are few, by instructions and reads of shared memory where they are many.  Measured on GB300, bf16, us a token
// forward: 8 heads of 64 x 64 0.30, 16 of 128 x 128 0.41, 128 of 128 x 128 1.8; the gradient's four walks 4.2 times that.
#include <algorithm>

#include "gated_delta.h"
#include "seq_common.cuh"

namespace prnn {
namespace {

constexpr int kThreads = 128, kLanes = 8, kCols = kThreads / kLanes;  // columns (rows) of one block
enum Walk { kValues = 0, kValueGrads = 1, kRowsForward = 2, kRowsBackward = 3 };

__device__ __forceinline__ float lanes8_sum(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Q: quads of one lane; the contracted axis has up to 32 Q values.
template <typename T, int WALK, int Q>
__global__ void __launch_bounds__(kThreads) gd_walk_kernel(const __grid_constant__ GdArgs a) {
  constexpr int N = 32 * Q, TB = Q > 4 ? 8 : 16, NV = WALK == kValues || WALK == kValueGrads ? 2 : 3;
  constexpr bool kRev = WALK == kValueGrads || WALK == kRowsBackward, kRows = WALK >= kRowsForward;
  constexpr int PER = NV * TB * N / kThreads;  // values a thread stages
  extern __shared__ __align__(16) float smem[];
  float* vec = smem;                           // [2][NV][TB][N]
  float* col = vec + 2 * NV * TB * N;          // [2][2][TB][kCols]
  float* gate = col + 4 * TB * kCols;          // [2][2][TB]
  float* res = gate + 4 * TB;                  // [2][TB][kCols]
  const int tid = threadIdx.x, lane = tid % kLanes, mine = tid / kLanes;
  const int c0 = blockIdx.y * kCols, c = c0 + mine;
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, hq = h / a.q.share;
  const int n = kRows ? a.dv : a.dk, m = kRows ? a.dk : a.dv;  // contracted axis, other axis
  int len = a.T;
  if (a.lens) {
    len = a.lens[b];
    len = len < 0 ? 0 : (len > a.T ? a.T : len);
  }
  const bool own = c < m;
  // value x of vector i of token t, and the two values that belong to one column
  auto vector = [&](int i, long long t, int x) -> float {
    if (x >= n) return 0.f;
    const long long row = ((t * a.B + b) * a.H + h) * a.dv + x;
    auto seq = [&](const LaSeq& s, int head) {
      return to_f32(static_cast<const T*>(s.p)[t * s.st + b * s.sb + head * s.sh + x]);
    };
    if (!kRows) return i == 0 ? seq(a.k, hq) : seq(a.q, hq);
    return i == 0 ? a.e[row] : (i == 1 ? a.du[row] : seq(a.d_o, h));
  };
  auto column = [&](int i, long long t, int cc) -> float {
    if (cc >= m) return 0.f;
    auto seq = [&](const LaSeq& s, int head) {
      return to_f32(static_cast<const T*>(s.p)[t * s.st + b * s.sb + head * s.sh + cc]);
    };
    if (WALK == kValues) return i == 0 ? seq(a.v, h) : 0.f;
    if (WALK == kValueGrads) return i == 0 ? seq(a.d_o, h) : 0.f;
    return i == 0 ? seq(a.k, hq) : (WALK == kRowsBackward ? seq(a.q, hq) : 0.f);
  };
  const int blocks = (len + TB - 1) / TB;
  constexpr int PERC = 2 * TB * kCols / kThreads;
  float staged[PER], staged_col[PERC], staged_gate;
  auto fetch = [&](int blk) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = j * kThreads + tid, x = i % N, t = blk * TB + i / N % TB;
      staged[j] = t < len ? vector(i / (N * TB), t, x) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < PERC; ++j) {
      const int i = j * kThreads + tid, t = blk * TB + i / kCols % TB;
      staged_col[j] = t < len ? column(i / (TB * kCols), t, c0 + i % kCols) : 0.f;
    }
    const long long t = blk * TB + tid % TB;
    staged_gate = 0.f;
    if (tid < 2 * TB && t < len)
      staged_gate = tid < TB ? a.g[t * a.gt + b * a.gb + h * a.gh] : a.beta[t * a.bt + b * a.bb + h * a.bh];
  };
  auto place = [&](int blk) {
    float* to = vec + (blk & 1) * NV * TB * N;
#pragma unroll
    for (int j = 0; j < PER; ++j) to[j * kThreads + tid] = staged[j];
#pragma unroll
    for (int j = 0; j < PERC; ++j) col[(blk & 1) * 2 * TB * kCols + j * kThreads + tid] = staged_col[j];
    if (tid < 2 * TB) gate[(blk & 1) * 2 * TB + tid] = tid < TB ? expf(staged_gate) : staged_gate;
  };
  // the state, transposed for walks over rows: this lane's quads of column (row) c
  float4 Z[Q];
  const float* from = WALK == kValues || WALK == kRowsForward ? a.state : a.d_state_out;
  const size_t head = (size_t)bh * a.dk * a.dv;
  auto at = [&](int x) { return head + (kRows ? (size_t)c * a.dv + x : (size_t)x * a.dv + c); };
#pragma unroll
  for (int j = 0; j < Q; ++j) {
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = (j * kLanes + lane) * 4 + i;
      z[i] = from && own && x < n ? from[at(x)] : 0.f;
    }
    Z[j] = make_float4(z[0], z[1], z[2], z[3]);
  }
  auto dot = [&](const float4 (&k)[Q]) {
    float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      s0 = fma2(make_float2(Z[j].x, Z[j].y), make_float2(k[j].x, k[j].y), s0);
      s1 = fma2(make_float2(Z[j].z, Z[j].w), make_float2(k[j].z, k[j].w), s1);
    }
    s0 = add2(s0, s1);
    return lanes8_sum(s0.x + s0.y);
  };
  auto update = [&](float f, float g, const float4 (&k)[Q]) {  // Z <- f Z + g k
    const float2 ff = both(f), gg = both(g);
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const float2 lo = fma2(gg, make_float2(k[j].x, k[j].y), mul2(ff, make_float2(Z[j].x, Z[j].y)));
      const float2 hi = fma2(gg, make_float2(k[j].z, k[j].w), mul2(ff, make_float2(Z[j].z, Z[j].w)));
      Z[j] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  };
  auto flush = [&](int blk) {
    for (int i = tid; i < TB * kCols; i += kThreads) {
      const long long t = blk * TB + i / kCols;
      const int cc = c0 + i % kCols;
      if (t >= len || cc >= m) continue;
      const float r0 = res[i], r1 = res[TB * kCols + i];
      const long long row = (t * a.B + b) * a.H + h;
      if (WALK == kValues) {
        if (a.e) a.e[row * a.dv + cc] = r0;
        if (a.o) static_cast<T*>(a.o)[t * a.ot + b * a.ob + h * a.oh + cc] = from_f32<T>(r1);
      } else if (WALK == kValueGrads) {
        a.du[row * a.dv + cc] = r0;
        if (a.dv_out) static_cast<T*>(a.dv_out)[t * a.dvt + b * a.dvb + h * a.dvh + cc] = from_f32<T>(r1);
      } else if (WALK == kRowsForward) {
        a.dk_part[row * a.dk + cc] = r0;
        a.dq_part[row * a.dk + cc] = r1;
      } else {
        a.dk_part[row * a.dk + cc] += r0;
      }
    }
  };
  // <S, R> at the end of a block of kGdBlock tokens: the walk over rows forwards leaves S, the one backwards meets it
  auto mark = [&](long long t) {
    float* keep = a.marks + ((size_t)(t / kGdBlock) * a.B * a.H + bh) * a.dk * a.dv + (size_t)c * a.dv;
    float s = 0.f;
    if (own)
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const float z[4] = {Z[j].x, Z[j].y, Z[j].z, Z[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = (j * kLanes + lane) * 4 + i;
          if (x >= n) continue;
          if (WALK == kRowsForward) keep[x] = z[i];
          else s = fmaf(z[i], keep[x], s);
        }
      }
    if (WALK == kRowsBackward) {
      s = lanes8_sum(s);
      if (own && lane == 0) a.leaves[((size_t)(t / kGdBlock) * a.B * a.H + bh) * a.dk + c] = s;
    }
  };
  if (blocks > 0) {
    fetch(kRev ? blocks - 1 : 0);
    place(kRev ? blocks - 1 : 0);
  }
  for (int i = 0; i < blocks; ++i) {
    const int blk = kRev ? blocks - 1 - i : i, next = kRev ? blk - 1 : blk + 1;
    if (i + 1 < blocks) fetch(next);
    __syncthreads();
    const float* v0 = vec + (blk & 1) * NV * TB * N;
    const float* s0 = col + (blk & 1) * 2 * TB * kCols;
    const float* g0 = gate + (blk & 1) * 2 * TB;
    const int live = min(TB, len - blk * TB);
    // a token's vectors and scalars, requested while the one before is worked on
    struct Token {
      float4 p[NV][Q];
      float x0, x1, dec, beta;
    } cur, ahead;
    constexpr bool kAhead = Q <= 4;  // wider ones have no registers for two
    auto take = [&](Token& to, int w) {
      const int t = kRev ? live - 1 - w : w;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < Q; ++j)
          to.p[v][j] = *reinterpret_cast<const float4*>(v0 + (v * TB + t) * N + (j * kLanes + lane) * 4);
      to.x0 = s0[t * kCols + mine];
      to.x1 = s0[(TB + t) * kCols + mine];
      to.dec = g0[t];
      to.beta = g0[TB + t];
    };
    if (kAhead) take(ahead, 0);
#pragma unroll 1
    for (int w = 0; w < live; ++w) {
      const int t = kRev ? live - 1 - w : w;
      const long long tt = (long long)blk * TB + t;
      if (kAhead) {
        cur = ahead;
        if (w + 1 < live) take(ahead, w + 1);
      } else {
        take(cur, w);
      }
      const float x0 = cur.x0, x1 = cur.x1, dec = cur.dec, beta = cur.beta;
      const float4 (&p0)[Q] = cur.p[0], (&p1)[Q] = cur.p[1], (&p2)[Q] = cur.p[NV - 1];
      float r0, r1 = 0.f;
      if (WALK == kValues) {
        r0 = fmaf(-dec, dot(p0), x0);
        update(dec, beta * r0, p0);
        r1 = a.o ? a.scale * dot(p1) : 0.f;
      } else if (WALK == kValueGrads) {
        update(1.f, a.scale * x0, p1);
        r0 = dot(p0);
        r1 = beta * r0;
        update(dec, -dec * r1, p0);
      } else if (WALK == kRowsForward) {
        r0 = -dec * beta * dot(p1);
        update(dec, beta * x0, p0);
        r1 = a.scale * dot(p2);
        if (tt == len - 1 || (tt + 1) % kGdBlock == 0) mark(tt);
      } else {
        if (tt == len - 1 || (tt + 1) % kGdBlock == 0) mark(tt);
        update(1.f, a.scale * x1, p2);
        r0 = beta * dot(p0);
        update(dec, -dec * beta * x0, p1);
      }
      if (lane == 0) {
        res[t * kCols + mine] = r0;
        res[(TB + t) * kCols + mine] = r1;
      }
    }
    __syncthreads();
    flush(blk);
    if (i + 1 < blocks) place(next);
  }
  float* to = WALK == kValues ? a.state_out : (WALK == kValueGrads ? a.d_state : nullptr);
  if (to && own)
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const float z[4] = {Z[j].x, Z[j].y, Z[j].z, Z[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = (j * kLanes + lane) * 4 + i;
        if (x < n) to[at(x)] = z[i];
      }
    }
  // zeros past the length
  if (WALK == kRowsForward)
    for (long long t = len + mine; t < a.T; t += kCols)
      for (int i = lane; i < kCols; i += kLanes)
        if (c0 + i < m) {
          const long long row = (t * a.B + b) * a.H + h;
          a.dq_part[row * a.dk + c0 + i] = 0.f;
          a.dk_part[row * a.dk + c0 + i] = 0.f;
        }
  if (kRows) return;
  T* out = static_cast<T*>(WALK == kValues ? a.o : a.dv_out);
  const long long st = WALK == kValues ? a.ot : a.dvt, sb = WALK == kValues ? a.ob : a.dvb,
                  sh = WALK == kValues ? a.oh : a.dvh;
  if (out)
    for (long long t = len + mine; t < a.T; t += kCols)
      for (int i = lane; i < kCols; i += kLanes)
        if (c0 + i < m) out[t * st + b * sb + h * sh + c0 + i] = from_f32<T>(0.f);
}

// The gates' gradients, a block of kGdBlock tokens at a time.
template <typename T>
__global__ void __launch_bounds__(256) gd_gates_kernel(const __grid_constant__ GdArgs a) {
  __shared__ float part[kGdBlock];
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int len = a.T;
  if (a.lens) {
    len = a.lens[b];
    len = len < 0 ? 0 : (len > a.T ? a.T : len);
  }
  for (long long blk = blockIdx.y; blk * kGdBlock < a.T; blk += gridDim.y) {
    const long long t0 = blk * kGdBlock;
    for (int i = warp; i < kGdBlock; i += 8) {
      const long long t = t0 + i;
      float s = 0.f, d = 0.f;
      if (t < len) {
        const long long row = (t * a.B + b) * a.H + h;
        const float beta = a.beta[t * a.bt + b * a.bb + h * a.bh];
        const T* q = static_cast<const T*>(a.q.p) + t * a.q.st + b * a.q.sb + (h / a.q.share) * a.q.sh;
        const T* v = static_cast<const T*>(a.v.p) + t * a.v.st + b * a.v.sb + h * a.v.sh;
        for (int x = lane; x < a.dk; x += 32) s = fmaf(to_f32(q[x]), a.dq_part[row * a.dk + x], s);
        float y = 0.f;
        for (int x = lane; x < a.dv; x += 32) {
          const float du = a.du[row * a.dv + x];
          y = fmaf(to_f32(v[x]), du, y);
          d = fmaf(a.e[row * a.dv + x], du, d);
        }
        s = warp_sum(fmaf(-beta, y, s));
        d = warp_sum(d);
      }
      if (lane == 0) {
        part[i] = s;
        if (t < a.T && a.dbeta) a.dbeta[t * a.dbt + b * a.dbb + h * a.dbh] = t < len ? d : 0.f;
      }
    }
    __syncthreads();
    if (a.dg && warp == 0) {
      float base = 0.f;
      if (t0 < len) {
        const float* leaves = a.leaves + ((size_t)blk * a.B * a.H + bh) * a.dk;
        for (int x = lane; x < a.dk; x += 32) base += leaves[x];
        base = warp_sum(base);
      }
      // sums from each token to the block's end: a lane's run of 4, then the runs after it
      constexpr int R = kGdBlock / 32;
      float s[R], run = 0.f;
#pragma unroll
      for (int i = R - 1; i >= 0; --i) s[i] = run += part[lane * R + i];
      float after = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float v = __shfl_down_sync(0xffffffffu, after, o);
        if (lane + o < 32) after += v;
      }
      after = __shfl_down_sync(0xffffffffu, after, 1);
      if (lane == 31) after = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const long long t = t0 + lane * R + i;
        if (t < a.T) a.dg[t * a.dgt + b * a.dgb + h * a.dgh] = t < len ? s[i] + after + base : 0.f;
      }
    }
    __syncthreads();
  }
}

template <typename T, int WALK, int Q>
cudaError_t walk(const GdArgs& a, cudaStream_t s) {
  constexpr int N = 32 * Q, TB = Q > 4 ? 8 : 16, NV = WALK <= kValueGrads ? 2 : 3;
  constexpr int smem = sizeof(float) * (2 * NV * TB * N + 4 * TB * kCols + 4 * TB + 2 * TB * kCols);
  auto kernel = gd_walk_kernel<T, WALK, Q>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int m = WALK >= kRowsForward ? a.dk : a.dv;
  kernel<<<dim3(a.B * a.H, (m + kCols - 1) / kCols), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int WALK>
cudaError_t walk(const GdArgs& a, cudaStream_t s) {
  const int n = WALK >= kRowsForward ? a.dv : a.dk;
  if (n <= 64) return walk<T, WALK, 2>(a, s);
  return n <= 128 ? walk<T, WALK, 4>(a, s) : walk<T, WALK, 8>(a, s);
}

}  // namespace

cudaError_t launch_gd_walk_forward(const GdArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  PRNN_BY_DTYPE(a.dtype, T, e = (walk<T, kValues>(a, s)));
  return e;
}

cudaError_t launch_gd_walk_backward(const GdArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  PRNN_BY_DTYPE(a.dtype, T, {
    if ((e = walk<T, kValues>(a, s)) != cudaSuccess) return e;
    if ((e = walk<T, kValueGrads>(a, s)) != cudaSuccess) return e;
    if ((e = walk<T, kRowsForward>(a, s)) != cudaSuccess) return e;
    if ((e = walk<T, kRowsBackward>(a, s)) != cudaSuccess) return e;
    const int blocks = (a.T + kGdBlock - 1) / kGdBlock;
    gd_gates_kernel<T><<<dim3(a.B * a.H, std::min(blocks, 65535)), 256, 0, s>>>(a);
  });
  return cudaGetLastError();
}

}  // namespace prnn
