// linear_attention.cu -- linear attention with a decay per head over whole
// sequences: the `mix` operation of seq_internal.h in all its roles, on CUDA cores,
// for any sizes, strides and types (fp32, and heads wider than 128).
//
// Unrolling S_t = l S_{t-1} + b_t c_t^T over a chunk of n tokens entered with
// state X gives
//   out_i = sum_{j<=i} l^(i-j) (a_i . b_j) c_j + l^(i+1) X^T a_i,
//   X'    = l^n X + sum_j l^(n-1-j) b_j c_j^T,
// so a chunk is four small matrix products and only the chunks are serial.
// Every exponent is >= 0: no power of the decay can overflow, whatever the
// decay, which factoring l^(i-j) into l^i l^-j would not give.
//
// Bound by the fp32 units in the limit (32-token chunks: 22 K multiply-adds per token and head at 128 x
// 128); what holds it at 0.24 of them is the latency of shared memory and loads at 16 warps an SM,
// which is what its tiles leave room for.  fp32 is kept to fp32 products: the tensor cores would need
// every operand in three 16-bit parts and six products.  Measured on GB300: T = 2048, 4 sequences of 16
// heads of 128 x 128 fp32 620 us (a plain one-column-slice kernel: 2984), T = 700, 5 sequences, 72 x
// 100 106 us (505).
#include "linear_attention_plan.h"
#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

constexpr int kChunk = 32, kCols = 64, kGroup = 128, kThreads = 2 * kGroup, kStride = kChunk + 4, kWide = kCols + 4;

struct SimtArgs {
  LaArgs g;
  int segs, cps, subs, cpb, slices, states_only;
  float* part;  // [role][B*H][subs][slices][D * kCols]
};

__device__ __forceinline__ int seq_len(const LaArgs& a, int b) {
  if (!a.lens) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

template <typename T>
__device__ __forceinline__ const T* seq_row(const LaSeq& s, long long t, int b, int h) {
  return static_cast<const T*>(s.p) + t * s.st + b * s.sb + (h / s.share) * s.sh;
}
// Four consecutive values of a row of n, zeros past it; `vec`: rows start on 16 bytes.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int at, int n, bool vec) {
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (vec && at + 4 <= n) {
    const Pack<T, 4> q = load_pack<T, 4>(p + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = to_f32(q.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j < n) v[j] = to_f32(p[at + j]);
  }
  return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// One block: one role, one (sequence, head), kCols of the e columns and one segment of time.  Both need
// only the chunk's tiles and the state before it, so half of the warps make the output while the other
// half make the scores, which the output needs last, and update the state.  The state stays in
// registers (thread (rg, cg): rows rg + 16 m, columns 4 cg .. and 32 + 4 cg ..) and is copied to shared
// memory once a chunk as an operand.  a and b are kept with the tokens innermost (a lane per token as
// they are loaded, so no bank conflicts), which serves the scores, the product with the state and the
// state's update: each product is a tile of 4 x 4 (scores 4 x 2, state 8 x 8) values per thread fed by
// 16-byte reads, 16 to 64 multiply-adds for two to four of them.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, D <= 64 ? 3 : (D <= 128 ? 2 : 1))
    la_simt_kernel(const __grid_constant__ SimtArgs args) {
  constexpr int M = D / 16;
  const LaArgs& g = args.g;
  const LaRole& r = g.role[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 31;
  const bool keeps_state = tid >= kGroup;       // the second group of warps; the first makes the output
  const int warp = (tid % kGroup) >> 5;         // within its group
  const int runs = args.states_only ? args.subs : args.segs;
  const int slice = blockIdx.x % args.slices, seg = blockIdx.x / args.slices % runs;
  const int bh = blockIdx.x / args.slices / runs, b = bh / g.H, h = bh % g.H;
  const int e0 = slice * kCols;
  if (e0 >= r.e) return;
  const int d = r.d, ncol = min(kCols, r.e - e0), len = seq_len(g, b);
  const int chunks = (len + kChunk - 1) / kChunk, last = len - (chunks - 1) * kChunk;
  const int per = args.states_only ? args.cpb : args.cps;
  const int from = min(seg * per, chunks), to = min((seg + 1) * per, chunks);
  auto before = [&](int c) {  // tokens processed before chunk c of the order
    if (c <= 0) return 0;
    if (c >= chunks) return len;
    return r.rev ? last + (c - 1) * kChunk : c * kChunk;
  };
  const bool with_out = !args.states_only && r.out;
  const bool writes_end = !args.states_only && r.x_end && (to > from ? to == chunks : chunks == 0 && seg == 0);
  if (with_out) {  // zeros past the length
    const int t0 = max(seg * per, chunks) * kChunk, t1 = min((seg + 1) * per * kChunk, g.T);
    for (long long p = tid; p < (long long)max(0, t1 - t0) * ncol; p += kThreads) {
      const long long at = (t0 + p / ncol) * r.ot + b * r.ob + h * r.oh + e0 + p % ncol;
      if (r.out_f32) static_cast<float*>(r.out)[at] = 0.f;
      else static_cast<T*>(r.out)[at] = from_f32<T>(0.f);
    }
  }
  if (to == from && !writes_end) return;

  extern __shared__ __align__(16) float sm[];
  float* At = sm;                    // [D][kStride]
  float* Bt = At + D * kStride;      // [D][kStride]
  float* Cs = Bt + D * kStride;      // [kChunk][kWide]
  float* Pt = Cs + kChunk * kWide;   // [kChunk (j)][kStride (i)]
  float* Xs = Pt + kChunk * kStride; // [D][kWide]
  __shared__ float pw[kChunk + 1];
  const float ld = g.log_decay[h];
  if (tid <= kChunk) pw[tid] = decay_pow(ld, tid);

  const int rg = warp * 4 + (lane >> 3), cg = lane & 7;  // the state's tile
  float X[M][8] = {};
  const size_t head = (size_t)bh * d * r.e;
  const int done = before(from);
  const float f0 = decay_pow(ld, done);
  if (keeps_state && r.x0 && !args.states_only)
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int k = rg + 16 * m, col = (c & 4) * 8 + 4 * cg + (c & 3);
      if (k < d && col < ncol)
        X[m][c] = f0 * r.x0[head + (r.x_t ? (size_t)(e0 + col) * d + k : (size_t)k * r.e + e0 + col)];
    }
  float* part = args.part + ((((size_t)blockIdx.y * g.B * g.H + bh) * args.subs) * args.slices + slice) * D * kCols;
  const size_t sub_size = (size_t)args.slices * D * kCols;
  if (keeps_state && !args.states_only) {
    const int subs = min(seg * (args.cps / args.cpb), (chunks + args.cpb - 1) / args.cpb);
    for (int u = 0; u < subs; ++u) {
      const float f = decay_pow(ld, done - before((u + 1) * args.cpb));
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(part + u * sub_size + (rg + 16 * m) * kCols + 32 * q + 4 * cg));
          X[m][4 * q] = fmaf(f, v.x, X[m][4 * q]);
          X[m][4 * q + 1] = fmaf(f, v.y, X[m][4 * q + 1]);
          X[m][4 * q + 2] = fmaf(f, v.z, X[m][4 * q + 2]);
          X[m][4 * q + 3] = fmaf(f, v.w, X[m][4 * q + 3]);
        }
    }
  }
  auto vec_of = [&](const LaSeq& s) {
    return (((reinterpret_cast<uintptr_t>(s.p) / sizeof(T)) | (uintptr_t)s.st | (uintptr_t)s.sb | (uintptr_t)s.sh) & 3) == 0;
  };
  const bool va = vec_of(r.a), vb = vec_of(r.b), vc = vec_of(r.c);
  const int r0 = 4 * (lane >> 2);                         // rows of the scores' and the output's tile
  const int pc = 8 * warp + 2 * (lane & 3), oc = 16 * warp + 4 * (lane & 3);  // their columns

  for (int ci = from; ci < to; ++ci) {
    const int t0 = (r.rev ? chunks - 1 - ci : ci) * kChunk, n = min(kChunk, len - t0);
    __syncthreads();
    if (with_out && keeps_state)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<float4*>(Xs + (rg + 16 * m) * kWide + 32 * q + 4 * cg) =
              make_float4(X[m][4 * q], X[m][4 * q + 1], X[m][4 * q + 2], X[m][4 * q + 3]);
    {
      const T* pa = seq_row<T>(r.a, t0 + lane, b, h);
      const T* pb = seq_row<T>(r.b, t0 + lane, b, h);
#pragma unroll 2
      for (int k = 4 * (tid >> 5); k < D; k += kThreads / 8) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (lane < n && k < d) {
          if (with_out) x = load4(pa, k, d, va);
          y = load4(pb, k, d, vb);
        }
        if (with_out) {
          At[k * kStride + lane] = x.x;
          At[(k + 1) * kStride + lane] = x.y;
          At[(k + 2) * kStride + lane] = x.z;
          At[(k + 3) * kStride + lane] = x.w;
        }
        Bt[k * kStride + lane] = y.x;
        Bt[(k + 1) * kStride + lane] = y.y;
        Bt[(k + 2) * kStride + lane] = y.z;
        Bt[(k + 3) * kStride + lane] = y.w;
      }
#pragma unroll
      for (int i = tid; i < kChunk * kCols / 4; i += kThreads) {
        const int j = i / (kCols / 4), c = i % (kCols / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < n) v = load4(seq_row<T>(r.c, t0 + j, b, h) + e0, c, ncol, vc);
        *reinterpret_cast<float4*>(Cs + j * kWide + c) = v;
      }
    }
    if (ci + 1 < to) {  // the next chunk on its way to L2 while this one is computed
      const int u0 = (r.rev ? chunks - 2 - ci : ci + 1) * kChunk, row = min(u0 + tid % kChunk, g.T - 1);
      const int at = tid / kChunk * (128 / (int)sizeof(T));  // a 128-byte line of the row per warp
      for (int k = at; k < d; k += kThreads / kChunk * (128 / (int)sizeof(T))) {
        if (with_out) prefetch_l2(seq_row<T>(r.a, row, b, h) + k);
        prefetch_l2(seq_row<T>(r.b, row, b, h) + k);
      }
      if (at < ncol) prefetch_l2(seq_row<T>(r.c, row, b, h) + e0 + at);
    }
    __syncthreads();
    if (with_out && !keeps_state) {
      float o[4][4] = {};
      auto product = [&](const float* x, int xstride, const float* y, int count) {
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
          const float4 u = ld4(x + k * xstride + r0), v = ld4(y + k * kWide + oc);
          const float us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = fmaf(us[i], vs[j], o[i][j]);
        }
      };
      product(At, kStride, Xs, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r0 + i, gap = (r.rev ? n - 1 - row : row) + r.lead;
        const float f = r.s_inter * pw[gap < 0 ? 0 : (gap > kChunk ? kChunk : gap)];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= f;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");  // the scores are there
      product(Pt, kStride, Cs, kChunk);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t0 + r0 + i >= g.T) break;
        const long long at = (long long)(t0 + r0 + i) * r.ot + b * r.ob + h * r.oh + e0 + oc;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (oc + j < ncol) {  // rows past the length: 0
            const float v = r0 + i < n ? o[i][j] : 0.f;
            if (r.out_f32) static_cast<float*>(r.out)[at + j] = v;
            else static_cast<T*>(r.out)[at + j] = from_f32<T>(v);
          }
      }
    }
    if (!keeps_state) continue;
    if (with_out) {
      // scores, weighted and masked
      float p[4][2] = {};
#pragma unroll 8
      for (int k = 0; k < d; ++k) {
        const float4 x = ld4(At + k * kStride + r0);
        const float2 y = *reinterpret_cast<const float2*>(Bt + k * kStride + pc);
        const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i][0] = fmaf(xs[i], y.x, p[i][0]);
          p[i][1] = fmaf(xs[i], y.y, p[i][1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int gap = r.rev ? pc + j - (r0 + i) : r0 + i - (pc + j);
          w[i] = gap >= 0 ? r.s_intra * p[i][j] * pw[gap] : 0.f;
        }
        *reinterpret_cast<float4*>(Pt + (pc + j) * kStride + r0) = make_float4(w[0], w[1], w[2], w[3]);
      }
      asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
    }
    // X <- l^n X + s_add sum_j w_j b_j c_j
    const float fn = pw[n];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int c = 0; c < 8; ++c) X[m][c] *= fn;
#pragma unroll 1
    for (int j = 0; j < kChunk; j += 4) {
      float bt[M][4];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float4 v = ld4(Bt + (rg + 16 * m) * kStride + j);
        bt[m][0] = v.x;
        bt[m][1] = v.y;
        bt[m][2] = v.z;
        bt[m][3] = v.w;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int gap = (r.rev ? j + q : n - 1 - j - q) + 1 - r.lead;
        const float w = j + q < n ? r.s_add * pw[gap] : 0.f;
        const float4 u = ld4(Cs + (j + q) * kWide + 4 * cg), v = ld4(Cs + (j + q) * kWide + 32 + 4 * cg);
        const float cw[8] = {w * u.x, w * u.y, w * u.z, w * u.w, w * v.x, w * v.y, w * v.z, w * v.w};
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int c = 0; c < 8; ++c) X[m][c] = fmaf(bt[m][q], cw[c], X[m][c]);
      }
    }
  }
  if (!keeps_state) return;
  if (writes_end)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int k = rg + 16 * m, col = (c & 4) * 8 + 4 * cg + (c & 3);
        if (k < d && col < ncol)
          r.x_end[head + (r.x_t ? (size_t)(e0 + col) * d + k : (size_t)k * r.e + e0 + col)] = X[m][c];
      }
  if (args.states_only)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float4*>(part + seg * sub_size + (rg + 16 * m) * kCols + 32 * q + 4 * cg) =
            make_float4(X[m][4 * q], X[m][4 * q + 1], X[m][4 * q + 2], X[m][4 * q + 3]);
}

template <typename T>
__global__ void __launch_bounds__(256) la_reduce_kernel(LaReduceArgs a) {
  const int hq = a.H / a.group;
  const long long n = (long long)a.T * a.B * hq * a.d;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const int k = (int)(i % a.d), h = (int)(i / a.d % hq), b = (int)(i / a.d / hq % a.B);
    const long long t = i / a.d / hq / a.B;
    const float* p = a.part + ((t * a.B + b) * a.H + (long long)h * a.group) * a.d + k;
    float s = 0.f;
    for (int j = 0; j < a.group; ++j) s += p[(long long)j * a.d];
    static_cast<T*>(a.out)[t * a.ot + b * a.ob + h * a.oh + k] = from_f32<T>(s);
  }
}

int max_d(const LaArgs& a) {
  int d = 0;
  for (int i = 0; i < a.roles; ++i) d = std::max(d, a.role[i].d);
  return d <= 64 ? 64 : (d <= 128 ? 128 : 256);
}
size_t smem_of(int D) {
  return sizeof(float) * (2 * D * kStride + kChunk * kWide + kChunk * kStride + D * kWide);
}
LaPlan make_plan(const LaArgs& a, size_t capacity) {
  const int D = max_d(a), at_once = std::min<int>(3, (int)(227 * 1024 / (smem_of(D) + 1024)));
  return la_plan(a, kChunk, kCols, at_once * seq_sm_count(), 0.45, sizeof(float) * D * kCols, capacity);
}

template <typename T, int D>
cudaError_t launch(SimtArgs& s, const LaPlan& p, cudaStream_t stream) {
  auto kernel = la_simt_kernel<T, D>;
  const size_t smem = smem_of(D);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const unsigned bh = (unsigned)(s.g.B * s.g.H * p.slices);
  if (p.segs > 1) {
    s.states_only = 1;
    kernel<<<dim3(bh * p.subs, s.g.roles), kThreads, smem, stream>>>(s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    s.states_only = 0;
  }
  kernel<<<dim3(bh * p.segs, s.g.roles), kThreads, smem, stream>>>(s);
  return cudaGetLastError();
}

}  // namespace

size_t la_simt_workspace(const LaArgs& a) {
  const LaPlan p = make_plan(a, ~(size_t)0);
  return sizeof(float) * a.roles * a.B * a.H * p.subs * p.slices * max_d(a) * kCols;
}

cudaError_t launch_la_simt(const LaArgs& a, void* scratch, size_t bytes, cudaStream_t stream) {
  if (a.roles == 0 || a.B == 0) return cudaSuccess;
  const LaPlan p = make_plan(a, bytes);
  SimtArgs s{a, p.segs, p.cps, p.subs, p.cpb, p.slices, 0, static_cast<float*>(scratch)};
  cudaError_t e = cudaSuccess;
  switch (max_d(a)) {
    case 64: PRNN_BY_DTYPE(a.dtype, T, (e = launch<T, 64>(s, p, stream))); break;
    case 128: PRNN_BY_DTYPE(a.dtype, T, (e = launch<T, 128>(s, p, stream))); break;
    default: PRNN_BY_DTYPE(a.dtype, T, (e = launch<T, 256>(s, p, stream))); break;
  }
  return e;
}

cudaError_t launch_la_reduce(const LaReduceArgs& a, cudaStream_t s) {
  const long long n = (long long)a.T * a.B * (a.H / a.group) * a.d;
  if (n == 0) return cudaSuccess;
  const long long want = (n + 255) / 256;
  const int blocks = (int)std::min<long long>(want, 16LL * seq_sm_count());
  PRNN_BY_DTYPE(a.dtype, T, (la_reduce_kernel<T><<<blocks, 256, 0, s>>>(a)));
  return cudaGetLastError();
}

}  // namespace prnn
