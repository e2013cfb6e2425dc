// rms_norm.cu -- root-mean-square norm over the last axis, with the residual's addition before it and an output
// in the data's type or in 8 bits (e4m3) with a scale per row or per 128 columns, and its gradient.
//
// Bound by memory: 5 to 9 flops per element against 4 to 16 bytes.  A row is read once and kept packed in
// registers, in its own type, between the sum of squares and the output: the stream is normalised as it is
// stored, so the packed form loses nothing and takes half the registers of fp32 values.  Blocks stay and request their
// next row while one is summed and written; two packs a thread measured best (8192 x 5760 bf16 into e4m3 83 us, with one
// pack 92, with four 112).  Measured on GB300, against the copy rate of 6.78 TB/s: 8192 x 4096 bf16 with residual 40 us (0.98),
// 8192 x 5760 with residual 63 (0.88) and into e4m3 81 (0.60: some 40 instructions a value where the other output takes 27, at
// 24 warps an SM), gradients with the stream's 8192 x 5760 fp32 121 (0.92), 8192 x 2304 fp32 58 and 7 to join dweight (0.68: a
// row's reduction stands between its loads and its store, and its blocks are one and a half waves, as said at their launch).
// Rows that 16-byte accesses do not fit go value by value: 8192 x 2001 bf16 with residual 70, into e4m3 115.
#include <algorithm>

#include <cuda_fp8.h>

#include "seq_common.cuh"
#include "seq_internal.h"

namespace prnn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kGroup = 128;           // columns of one scale
constexpr int kMostGroups = 8192 / kGroup;

// NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// Over groups of N neighbouring lanes, N a power of two up to 32.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float block_max(float v, float* part) {
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  v = lanes_max<32>(v);
  if ((threadIdx.x & 31) == 0) part[warp] = v;
  __syncthreads();
  float m = part[0];
  for (int w = 1; w < warps; ++w) m = max_nan(m, part[w]);
  return m;
}
// A group of zeros has the scale 1, and so has one so small that its scale's inverse leaves fp32's range.
constexpr float kLeastTop = 7.888609e-31f;  // 2^-100
__device__ __forceinline__ float scale_of(float top) { return top > kLeastTop ? top * (1.f / kE4m3Max) : 1.f; }
// What a value is multiplied by instead of divided by its scale: a rounding of 2^-24 more before that of 2^-4.
__device__ __forceinline__ float inverse_of(float top) { return top > kLeastTop ? kE4m3Max / top : 1.f; }
__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

template <int V>
__device__ __forceinline__ Pack<float, V> weights(const float* w, int c) {
  Pack<float, V> r;
  if (!w) {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = 1.f;
  } else if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(r.v + i) = __ldg(reinterpret_cast<const float4*>(w + c + i));
  } else {
    r.v[0] = __ldg(w + c);
  }
  return r;
}

// x + residual, rounded to T.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> added(const Pack<T, V>& x, const Pack<T, V>& r) {
  Pack<T, V> h;
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) set_pair<T, V>(h, i, add2(pair_of<T, V>(x, i), pair_of<T, V>(r, i)));
  return h;
}
template <typename T, int V>
__device__ __forceinline__ float squares(const Pack<T, V>& h) {
  float2 acc = both(0.f);
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) {
    const float2 f = pair_of<T, V>(h, i);
    acc = fma2(f, f, acc);
  }
  return acc.x + acc.y;
}
template <typename T, int V>
__device__ __forceinline__ Pack<float, V> normed(const Pack<T, V>& h, float rstd, const Pack<float, V>& w) {
  Pack<float, V> y;
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i)
    set_pair<float, V>(y, i, mul2(mul2(pair_of<T, V>(h, i), both(rstd)), pair_of<float, V>(w, i)));
  return y;
}
template <int V>
__device__ __forceinline__ float top_of(const Pack<float, V>& y) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max_nan(m, fabsf(y.v[i]));
  return m;
}
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* q, const Pack<float, V>& y, float inverse) {
  if constexpr (V == 1) {
    *q = to_e4m3(y.v[0] * inverse);
  } else {
    Pack<uint16_t, V / 2> o;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      o.v[i] = (uint16_t)__nv_cvt_float2_to_fp8x2(mul2(pair_of<float, V>(y, i), both(inverse)), __NV_SATFINITE, __NV_E4M3);
    store_pack<uint16_t, V / 2>(reinterpret_cast<uint16_t*>(q), o);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_y(T* y, const Pack<float, V>& f) {
  Pack<T, V> o;
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) set_pair<T, V>(o, i, pair_of<float, V>(f, i));
  store_pack<T, V>(y, o);
}

// What a thread holds of a row before the residual's addition: the packs t, t + width, ... of V columns.
template <typename T, int V, int NV>
struct RowPacks {
  Pack<T, V> x[NV], res[NV];
  __device__ __forceinline__ void load(const RmsNormArgs& a, long long r, int t, int width) {
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int c = (p * width + t) * V;
      if (r >= a.rows || c >= a.cols) continue;
      x[p] = load_once<T, V>(static_cast<const T*>(a.x) + r * a.x_stride + c);
      if (a.residual) res[p] = load_once<T, V>(static_cast<const T*>(a.residual) + r * a.residual_stride + c);
    }
  }
};

// One row.  TPR > 0: TPR neighbouring lanes hold it (no barrier; lanes without a row go along with `live`
// false); TPR == 0: the whole block does.
template <typename T, int V, int NV, int TPR, bool Q>
__device__ __forceinline__ void rms_row(const RmsNormArgs& a, RowPacks<T, V, NV>& in, long long r, bool live, int t,
                                        int width, float* part, unsigned* tops) {
  const bool res = a.residual != nullptr;
  Pack<T, V> (&h)[NV] = in.x;
  float s = 0.f;
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    const int c = (p * width + t) * V;
    if (!live || c >= a.cols) continue;
    if (res) {
      h[p] = added<T, V>(h[p], in.res[p]);
      store_pack<T, V>(static_cast<T*>(a.h) + r * a.h_stride + c, h[p]);
    }
    s += squares<T, V>(h[p]);
  }
  if constexpr (TPR > 0) s = lanes_sum<TPR>(s);
  else s = block_sum(s, part);
  const float rstd = 1.f / sqrtf(s / a.cols + a.eps);
  if (live && t == 0 && a.rstd) a.rstd[r] = rstd;
  if constexpr (!Q) {
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int c = (p * width + t) * V;
      if (live && c < a.cols)
        store_y<T, V>(static_cast<T*>(a.y) + r * a.y_stride + c, normed<T, V>(h[p], rstd, weights<V>(a.weight, c)));
    }
  } else {
    Pack<float, V> y[NV];
    float top[NV];
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int c = (p * width + t) * V;
      top[p] = 0.f;
      if (live && c < a.cols) {
        y[p] = normed<T, V>(h[p], rstd, weights<V>(a.weight, c));
        top[p] = top_of<V>(y[p]);
      }
    }
    const int groups = a.group ? (a.cols + a.group - 1) / a.group : 1;
    float* scale = a.scale + r * groups;
    if (!a.group || groups == 1) {  // one scale for the row
      float m = top[0];
#pragma unroll
      for (int p = 1; p < NV; ++p) m = max_nan(m, top[p]);
      if constexpr (TPR > 0) m = lanes_max<TPR>(m);
      else m = block_max(m, part + 32);
#pragma unroll
      for (int p = 0; p < NV; ++p) top[p] = m;
      if (live && t == 0) scale[0] = scale_of(m);
    } else if constexpr (V > 1) {
      // 128 columns lie in 128 / V neighbouring lanes
      constexpr int N = TPR > 0 && TPR < kGroup / V ? TPR : kGroup / V;
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int c = (p * width + t) * V;
        top[p] = lanes_max<N>(top[p]);
        if (live && c < a.cols && c % kGroup == 0) scale[c / kGroup] = scale_of(top[p]);
      }
    } else if constexpr (TPR == 0) {
      // single columns: a warp's 32 lie in one group, whose maximum is that of its warps (as the bits of
      // values that are not negative, the largest whatever the order)
      for (int g = t; g < groups; g += width) tops[g] = 0u;
      __syncthreads();
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const float m = lanes_max<32>(top[p]);
        const int c = (p * width + t) & ~31;
        if ((t & 31) == 0 && c < a.cols) atomicMax(&tops[c / kGroup], __float_as_uint(m));
      }
      __syncthreads();
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int c = p * width + t;
        if (c < a.cols) top[p] = __uint_as_float(tops[c / kGroup]);
        if (c < a.cols && c % kGroup == 0) scale[c / kGroup] = scale_of(top[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int c = (p * width + t) * V;
      if (live && c < a.cols)
        store_e4m3<V>(static_cast<uint8_t*>(a.y) + r * a.y_stride + c, y[p], inverse_of(top[p]));
    }
  }
}

// A row per block.  Four packs of values in fp32 before they are rounded to 8 bits take more registers than
// 1024 threads have; the other output takes the same plan, so that both have the same sums.
template <int NV>
constexpr int kMostThreads = NV == 4 ? 512 : 1024;
template <typename T, int V, int NV, bool Q>
__global__ void __launch_bounds__(kMostThreads<NV>) rms_block_kernel(RmsNormArgs a) {
  __shared__ float part[2][64];
  __shared__ unsigned tops[Q && V == 1 ? kMostGroups : 1];
  RowPacks<T, V, NV> cur, ahead;
  cur.load(a, blockIdx.x, threadIdx.x, blockDim.x);
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    ahead.load(a, r + gridDim.x, threadIdx.x, blockDim.x);
    rms_row<T, V, NV, 0, Q>(a, cur, r, true, threadIdx.x, blockDim.x, part[turn], tops);
    if (Q && V == 1) __syncthreads();
    cur = ahead;
  }
}
// A row per TPR lanes.
template <typename T, int V, int NV, int TPR, bool Q>
__global__ void __launch_bounds__(256) rms_lanes_kernel(RmsNormArgs a) {
  const long long r = (long long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  RowPacks<T, V, NV> in;
  in.load(a, r, threadIdx.x % TPR, TPR);
  rms_row<T, V, NV, TPR, Q>(a, in, r, r < a.rows, threadIdx.x % TPR, TPR, nullptr, nullptr);
}

// Rows too long for registers: a block per row, which is read again (from L2) for each step.  Columns are counted
// in 64 bits: a step past the last of nearly 2^31 does not fit 32.
template <typename T, bool Q>
__global__ void __launch_bounds__(1024) rms_long_kernel(RmsNormArgs a) {
  __shared__ float part[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + r * a.residual_stride : nullptr;
    const T* h = res ? static_cast<const T*>(a.h) + r * a.h_stride : x;
    float s = 0.f;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) {
      float f = to_f32(x[c]);
      if (res) {
        const T sum = from_f32<T>(f + to_f32(res[c]));
        static_cast<T*>(a.h)[r * a.h_stride + c] = sum;
        f = to_f32(sum);
      }
      s = fmaf(f, f, s);
    }
    const float rstd = 1.f / sqrtf(block_sum(s, part[0]) / a.cols + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    auto value = [&](long long c) { return to_f32(h[c]) * rstd * (a.weight ? a.weight[c] : 1.f); };
    if constexpr (!Q) {
      T* y = static_cast<T*>(a.y) + r * a.y_stride;
      for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) y[c] = from_f32<T>(value(c));
    } else {
      // a group per warp; the thread that wrote a stream's value is not the one that reads it
      __syncthreads();
      uint8_t* q = static_cast<uint8_t*>(a.y) + r * a.y_stride;
      if (a.group) {
        const long long groups = ((long long)a.cols + a.group - 1) / a.group;
        for (long long g = warp; g < groups; g += warps) {
          float v[kGroup / 32], top = 0.f;
#pragma unroll
          for (int i = 0; i < kGroup / 32; ++i) {
            const long long c = g * kGroup + i * 32 + lane;
            v[i] = c < a.cols ? value(c) : 0.f;
            top = max_nan(top, fabsf(v[i]));
          }
          top = lanes_max<32>(top);
          if (lane == 0) a.scale[r * groups + g] = scale_of(top);
          const float inverse = inverse_of(top);
#pragma unroll
          for (int i = 0; i < kGroup / 32; ++i) {
            const long long c = g * kGroup + i * 32 + lane;
            if (c < a.cols) q[c] = to_e4m3(v[i] * inverse);
          }
        }
      } else {
        float top = 0.f;
        for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) top = max_nan(top, fabsf(value(c)));
        top = block_max(top, part[1]);
        if (threadIdx.x == 0) a.scale[r] = scale_of(top);
        const float inverse = inverse_of(top);
        for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) q[c] = to_e4m3(value(c) * inverse);
      }
    }
    __syncthreads();
  }
}

constexpr int kRmsOne = 128, kRmsTwo = 512;  // threads of one and two packs each, where rows are many

template <typename T, int V, bool Q>
void launch_forward(const RmsNormArgs& a, cudaStream_t s) {
  const int packs = (a.cols + V - 1) / V;
  auto lanes = [&](auto kernel, int tpr) {
    kernel<<<(unsigned)((a.rows + 256 / tpr - 1) / (256 / tpr)), 256, 0, s>>>(a);
  };
  const bool one = (a.rows + 7) / 8 <= 0x7fffffff;  // a grid has as many blocks
  if (one && V > 1 && packs <= 8) return lanes(rms_lanes_kernel<T, V, 1, 8, Q>, 8);
  if (one && V > 1 && packs <= 16) return lanes(rms_lanes_kernel<T, V, 1, 16, Q>, 16);
  if (one && V > 1 && packs <= 32) return lanes(rms_lanes_kernel<T, V, 1, 32, Q>, 32);
  if (one && V == 1 && packs <= 128) return lanes(rms_lanes_kernel<T, V, V == 1 ? 4 : 1, 32, Q>, 32);
  // With few rows a row is spread over as many threads as it has packs; with many, blocks stay and go on to a row a
  // grid away, whose loads are under way while this one is summed and written.
  const bool many = a.rows >= 4LL * seq_sm_count();
  auto threads = [&](int nv) { return ((packs + nv - 1) / nv + 31) / 32 * 32; };
  auto block = [&](auto kernel, int nv) {
    // as many blocks as an SM holds by (a bound on) their registers, no part of another wave
    const int regs = V == 1 ? (nv > 4 ? 64 : 48) : (nv == 1 ? 56 : (nv == 4 ? 128 : (V == 8 && !Q ? 56 : 64)));
    const int n = threads(nv), per_sm = std::max(1, std::min(2048, 65536 / regs) / n);
    kernel<<<(unsigned)std::min<long long>(a.rows, (long long)per_sm * seq_sm_count()), n, 0, s>>>(a);
  };
  if (threads(1) <= (many ? kRmsOne : 1024)) {
    block(rms_block_kernel<T, V, 1, Q>, 1);
  } else if (threads(2) <= (many ? kRmsTwo : 1024)) {
    block(rms_block_kernel<T, V, 2, Q>, 2);
  } else if (threads(4) <= kMostThreads<4>) {
    block(rms_block_kernel<T, V, 4, Q>, 4);
  } else if (V == 1 && threads(8) <= 1024) {
    block(rms_block_kernel<T, V, V == 1 ? 8 : 1, Q>, 8);
  } else {
    rms_long_kernel<T, Q><<<(unsigned)std::min<long long>(a.rows, 4LL * seq_sm_count()), 1024, 0, s>>>(a);
  }
}

bool fits(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---- gradient -------------------------------------------------------------------------------------
// dx = rstd (g - xhat mean(g xhat)) + dh, g = dy w, xhat = h rstd; dw = sum over rows of dy xhat.  Blocks
// visit rows a grid apart and keep their part of dw in registers; the parts are joined in order.

// A row per turn of TPR lanes (0: of the block), the next row's values requested before the sum.
template <typename T, int V, int NV, int TPR>
__device__ __forceinline__ void rms_grad_rows(const RmsNormGradArgs& a, long long first, long long step, int t,
                                              int width, float (*part)[32], Pack<float, V> (&dw)[NV]) {
  struct Row {
    Pack<T, V> h[NV], dy[NV], dh[NV];
    float rstd;
  };
  auto load = [&](Row& x, long long r) {
    const bool in = r < a.rows;
    x.rstd = in ? __ldg(a.rstd + r) : 0.f;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int c = (p * width + t) * V;
      if (!in || c >= a.cols) continue;
      x.h[p] = load_once<T, V>(static_cast<const T*>(a.h) + r * a.h_stride + c);
      x.dy[p] = load_once<T, V>(static_cast<const T*>(a.dy) + r * a.dy_stride + c);
      if (a.dh) x.dh[p] = load_once<T, V>(static_cast<const T*>(a.dh) + r * a.dh_stride + c);
    }
  };
  // The weights stay in registers where the rows leave room for them, else they come from L1 each time.
  constexpr bool kKeep = NV * V <= 16;
  constexpr bool kAhead = NV * V <= 16;
  Pack<float, V> w[kKeep ? NV : 1];
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    const int c = (p * width + t) * V;
    if (kKeep && c < a.cols) w[p] = weights<V>(a.weight, c);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[p].v[i] = 0.f;
  }
  auto weight = [&](int p, int c) {
    if constexpr (kKeep) return w[p];
    else return weights<V>(a.weight, c);
  };
  Row cur;
  load(cur, first);
  int turn = 0;
  // every lane of a warp makes the same number of turns
  for (long long r0 = first - (TPR > 0 && TPR < 32 ? (threadIdx.x & 31) / (TPR ? TPR : 1) : 0); r0 < a.rows;
       r0 += step, ++turn) {
    const long long r = first + turn * step;
    const bool live = r < a.rows;
    Row next;
    if (kAhead) load(next, r + step);
    float s = 0.f;
    if (live)
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int c = (p * width + t) * V;
        if (c >= a.cols) continue;
        const Pack<float, V> wp = weight(p, c);
        float2 acc = both(0.f);
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) {
          const float2 xhat = mul2(pair_of<T, V>(cur.h[p], i), both(cur.rstd)), dy = pair_of<T, V>(cur.dy[p], i);
          acc = fma2(mul2(dy, pair_of<float, V>(wp, i)), xhat, acc);
          set_pair<float, V>(dw[p], i, fma2(dy, xhat, pair_of<float, V>(dw[p], i)));
        }
        s += acc.x + acc.y;
      }
    if constexpr (TPR > 0) s = lanes_sum<TPR>(s);
    else s = block_sum(s, part[turn & 1]);
    const float mean = s / a.cols;
    if (live && a.dx)
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int c = (p * width + t) * V;
        if (c >= a.cols) continue;
        const Pack<float, V> wp = weight(p, c);
        Pack<T, V> o;
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) {
          const float2 xhat = mul2(pair_of<T, V>(cur.h[p], i), both(cur.rstd));
          const float2 g = mul2(pair_of<T, V>(cur.dy[p], i), pair_of<float, V>(wp, i));
          float2 d = mul2(both(cur.rstd), fma2(xhat, both(-mean), g));
          if (a.dh) d = add2(d, pair_of<T, V>(cur.dh[p], i));
          set_pair<T, V>(o, i, d);
        }
        store_pack<T, V>(static_cast<T*>(a.dx) + r * a.dx_stride + c, o);
      }
    if (kAhead) cur = next;
    else load(cur, r + step);
  }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(512) rms_grad_block_kernel(RmsNormGradArgs a) {
  __shared__ float part[2][32];
  Pack<float, V> dw[NV];
  rms_grad_rows<T, V, NV, 0>(a, blockIdx.x, gridDim.x, threadIdx.x, blockDim.x, part, dw);
  if (!a.dweight) return;
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * V;
    if (c < a.cols)
#pragma unroll
      for (int i = 0; i < V; ++i) a.partial[(size_t)blockIdx.x * a.cols + c + i] = dw[p].v[i];
  }
}

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(256) rms_grad_lanes_kernel(RmsNormGradArgs a) {
  constexpr int R = 256 / TPR, W = TPR * NV * V;
  __shared__ float sums[R][W + 1];
  Pack<float, V> dw[NV];
  const int t = threadIdx.x % TPR, mine = threadIdx.x / TPR;
  rms_grad_rows<T, V, NV, TPR>(a, (long long)blockIdx.x * R + mine, (long long)gridDim.x * R, t, TPR, nullptr, dw);
  if (!a.dweight) return;
#pragma unroll
  for (int p = 0; p < NV; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) sums[mine][(p * TPR + t) * V + i] = dw[p].v[i];
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += 256) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) s += sums[i][c];
    a.partial[(size_t)blockIdx.x * a.cols + c] = s;
  }
}

__global__ void __launch_bounds__(1024) rms_join_kernel(const float* partial, int splits, int cols, float* dweight) {
  __shared__ float sums[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  for (long long c0 = 32LL * blockIdx.x; c0 < cols; c0 += 32LL * gridDim.x) {
    const long long c = c0 + tx;
    float s = 0.f;
    if (c < cols)
#pragma unroll 4
      for (int i = ty; i < splits; i += 32) s += partial[(size_t)i * cols + c];
    sums[ty][tx] = s;
    __syncthreads();
    s = warp_sum(sums[tx][ty]);
    if (tx == 0 && c0 + ty < cols) dweight[c0 + ty] = s;
    __syncthreads();
  }
}

// Rows too long for registers: the columns' sums a thread each, then dx by rows.  Both read dy.
template <typename T>
__global__ void __launch_bounds__(1024) rms_dx_long_kernel(RmsNormGradArgs a) {
  __shared__ float part[32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *h = static_cast<const T*>(a.h) + r * a.h_stride, *dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + r * a.dh_stride : nullptr;
    T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
    const float rstd = a.rstd[r];
    float s = 0.f;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x)
      s = fmaf(to_f32(dy[c]) * (a.weight ? a.weight[c] : 1.f), to_f32(h[c]) * rstd, s);
    const float mean = block_sum(s, part) / a.cols;
    for (long long c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(dy[c]) * (a.weight ? a.weight[c] : 1.f);
      float d = rstd * fmaf(to_f32(h[c]) * rstd, -mean, g);
      if (dh) d += to_f32(dh[c]);
      dx[c] = from_f32<T>(d);
    }
    __syncthreads();
  }
}
template <typename T>
__global__ void __launch_bounds__(256) rms_dw_long_kernel(RmsNormGradArgs a, int splits) {
  const long long each = (a.rows + splits - 1) / splits, lo = blockIdx.y * each,
                  hi = lo + each < a.rows ? lo + each : a.rows;
  for (long long c = blockIdx.x * 256LL + threadIdx.x; c < a.cols; c += gridDim.x * 256LL) {
    float s = 0.f;
    for (long long r = lo; r < hi; ++r)
      s = fmaf(to_f32(static_cast<const T*>(a.dy)[r * a.dy_stride + c]),
               to_f32(static_cast<const T*>(a.h)[r * a.h_stride + c]) * a.rstd[r], s);
    a.partial[(size_t)blockIdx.y * a.cols + c] = s;
  }
}

template <typename T, int V>
cudaError_t launch_backward(RmsNormGradArgs a, int splits, cudaStream_t s) {
  const int packs = (a.cols + V - 1) / V;
  // As many blocks as the SMs hold at once by their registers: up to 72 a thread in most kernels of up to 8 values, 80 in
  // blocks of 256 threads, which are three an SM either way, and 128 for more values.  A part of another wave costs more
  // than it adds (32768 x 1152 bf16: with 5 an SM 67 us, with 8 75, with 6 90, with 4 124).  Two kernels hold more than
  // is taken here, and some widths get up to twice the blocks that fit: fp32 in two packs of four (110 registers, 1025 to 3584
  // columns; 2304 columns are three blocks of 288 threads an SM where two fit), and four single values a thread (78 in bf16
  // and 84 in fp32, widths among 1025 to 1792).
  auto resident = [&](int nv, int threads) { return std::max(1, 65536 / ((nv * V <= 8 ? 72 : 128) * threads)); };
  auto lanes = [&](auto kernel, int tpr) {
    const int rows = 256 / tpr;
    splits = (int)std::min<long long>({splits, (a.rows + rows - 1) / rows, resident(1, 256) * (long long)seq_sm_count()});
    kernel<<<splits, 256, 0, s>>>(a);
  };
  auto threads = [&](int nv) { return ((packs + nv - 1) / nv + 31) / 32 * 32; };
  auto block = [&](auto kernel, int nv) {
    splits = std::min(splits, resident(nv, threads(nv)) * seq_sm_count());
    kernel<<<splits, threads(nv), 0, s>>>(a);
  };
  if (V > 1 && packs <= 8) {
    lanes(rms_grad_lanes_kernel<T, V, 1, 8>, 8);
  } else if (V > 1 && packs <= 16) {
    lanes(rms_grad_lanes_kernel<T, V, 1, 16>, 16);
  } else if (V > 1 && packs <= 32) {
    lanes(rms_grad_lanes_kernel<T, V, 1, 32>, 32);
  } else if (V == 1 && packs <= 128) {
    lanes(rms_grad_lanes_kernel<T, V, V == 1 ? 4 : 1, 32>, 32);
  } else if (threads(1) <= 256) {
    block(rms_grad_block_kernel<T, V, 1>, 1);
  } else if (threads(2) <= 512) {
    block(rms_grad_block_kernel<T, V, 2>, 2);
  } else if (V > 1 && threads(4) <= 512) {
    block(rms_grad_block_kernel<T, V, (V > 1 ? 4 : 1)>, 4);
  } else if (V == 1 && threads(4) <= 512) {
    block(rms_grad_block_kernel<T, V, V == 1 ? 4 : 1>, 4);
  } else if (V == 1 && threads(8) <= 512) {
    block(rms_grad_block_kernel<T, V, V == 1 ? 8 : 1>, 8);
  } else if (V == 1 && threads(16) <= 512) {
    block(rms_grad_block_kernel<T, V, V == 1 ? 16 : 1>, 16);
  } else {
    if (a.dweight) {  // before dx, which may be written over dy
      const unsigned gx = (unsigned)std::min<long long>((a.cols + 255LL) / 256, 65535);
      rms_dw_long_kernel<T><<<dim3(gx, splits), 256, 0, s>>>(a, splits);
    }
    if (a.dx)
      rms_dx_long_kernel<T><<<(unsigned)std::min<long long>(a.rows, 4LL * seq_sm_count()), 1024, 0, s>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dweight) return e;
  rms_join_kernel<<<(unsigned)std::min<long long>((a.cols + 31LL) / 32, 65535), 1024, 0, s>>>(a.partial, splits, a.cols,
                                                                                             a.dweight);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t s) {
  const int v = a.dtype == PRNN_F32 ? 4 : 8;
  const bool rows = a.rows > 1;
  auto row_ok = [&](const void* p, long long stride, size_t align) {
    return !p || (fits(p, align) && (!rows || stride % v == 0));
  };
  const bool vec = a.cols % v == 0 && row_ok(a.x, a.x_stride, 16) && row_ok(a.residual, a.residual_stride, 16) &&
                   row_ok(a.h, a.h_stride, 16) && row_ok(a.y, a.y_stride, a.scale ? v : 16) && fits(a.weight, 16);
  PRNN_BY_DTYPE(a.dtype, T, {
    constexpr int V = 16 / sizeof(T);
    if (a.scale) vec ? launch_forward<T, V, true>(a, s) : launch_forward<T, 1, true>(a, s);
    else vec ? launch_forward<T, V, false>(a, s) : launch_forward<T, 1, false>(a, s);
  });
  return cudaGetLastError();
}

// Blocks whose parts of dweight are kept apart, at most: enough for every type's plan.
int rms_norm_splits(long long rows, int cols) {
  const long long per_sm = cols <= 1024 ? 10 : (cols <= 4096 ? 5 : 2);
  return (int)std::max(1LL, std::min(rows, per_sm * seq_sm_count()));
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, cudaStream_t s) {
  const int v = a.dtype == PRNN_F32 ? 4 : 8;
  const bool rows = a.rows > 1;
  auto row_ok = [&](const void* p, long long stride) { return !p || (fits(p, 16) && (!rows || stride % v == 0)); };
  const bool vec = a.cols % v == 0 && row_ok(a.dy, a.dy_stride) && row_ok(a.h, a.h_stride) &&
                   row_ok(a.dh, a.dh_stride) && row_ok(a.dx, a.dx_stride) && fits(a.weight, 16);
  const int splits = rms_norm_splits(a.rows, a.cols);
  cudaError_t e = cudaSuccess;
  PRNN_BY_DTYPE(a.dtype, T, {
    constexpr int V = 16 / sizeof(T);
    e = vec ? launch_backward<T, V>(a, splits, s) : launch_backward<T, 1>(a, splits, s);
  });
  return e;
}

}  // namespace prnn
