// seq_checks.h -- checks of arguments that the C ABI functions of the sequence operators share: types,
// alignment, the extents of strided tensors and whether outputs overlap anything.
#pragma once

#include <algorithm>
#include <climits>
#include <cstdint>

#include "host_util.h"
#include "prnn.h"
#include "seq_internal.h"

namespace prnn {

inline size_t elem_size(prnn_dtype_t d) { return d == PRNN_F32 ? 4 : 2; }
inline bool known(prnn_dtype_t d) { return d == PRNN_F32 || d == PRNN_F16 || d == PRNN_BF16; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Elements from the first to the last of `rows` rows; -1 when that is no size.
inline long long row_extent(long long rows, long long cols, long long stride) {
  if (rows <= 0) return 0;
  long long v;
  if (__builtin_mul_overflow(rows - 1, stride, &v) || __builtin_add_overflow(v, cols, &v) ||
      v > LLONG_MAX / 8)
    return -1;
  return v;
}

// A sequence tensor's dimensions with their strides, outermost stride first.
struct Dims {
  long long n[3], s[3];
  int w;  // values of the contiguous last axis
};
inline Dims dims_of(const prnn_seq_t& x, int T, int B, int H, int w) {
  Dims d{{T, B, H}, {x.stride_t, x.stride_b, x.stride_h}, w};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (d.s[j] > d.s[i]) {
        std::swap(d.s[i], d.s[j]);
        std::swap(d.n[i], d.n[j]);
      }
  return d;
}
// Elements spanned by the dimensions from `from` inwards; -1 on overflow.
inline long long span(const Dims& d, int from) {
  long long v = d.w;
  for (int i = from; i < 3; ++i) {
    long long m;
    if (__builtin_mul_overflow(d.n[i] - 1, d.s[i], &m) || __builtin_add_overflow(v, m, &v) ||
        v > LLONG_MAX / 8)
      return -1;
  }
  return v;
}
// Every element of an output has an address of its own.
inline bool distinct(const Dims& d) {
  for (int i = 0; i < 3; ++i)
    if (d.n[i] > 1 && d.s[i] < span(d, i + 1)) return false;
  return true;
}
// Two tensors share no element: their spans are apart, or they lie beside one another in a
// joint layout (equal strides, each within a part of the same period).
inline bool apart(const void* pa, const Dims& a, const void* pb, const Dims& b, size_t esz) {
  if (!overlaps(pa, (size_t)span(a, 0) * esz, pb, (size_t)span(b, 0) * esz)) return true;
  const long long byte = static_cast<const char*>(pa) - static_cast<const char*>(pb);
  if (byte % (long long)esz != 0) return false;
  const long long off = byte / (long long)esz;
  for (int i = 0; i < 3; ++i) {
    if (a.s[i] != b.s[i] || a.s[i] <= 0) return false;
    bool period = true;
    for (int j = 0; j < i; ++j) period = period && a.s[j] % a.s[i] == 0;
    if (!period) continue;
    const long long m = ((off % a.s[i]) + a.s[i]) % a.s[i];
    if (m >= span(b, i + 1) && m + span(a, i + 1) <= a.s[i]) return true;
  }
  return false;
}

// An input or output of one call, for the checks.
struct Part {
  const void* p;
  Dims d;
  bool out;
};
inline bool seq_ok(const prnn_seq_t& x, const Dims& d, size_t esz, bool out) {
  return x.data && aligned(x.data, esz) && x.stride_t >= 0 && x.stride_b >= 0 && x.stride_h >= 0 &&
         span(d, 0) > 0 && (!out || distinct(d));
}
inline bool outputs_apart(const Part* part, int n, size_t esz) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (i != j && part[i].out && (!part[j].out || i < j) &&
          !apart(part[i].p, part[i].d, part[j].p, part[j].d, esz))
        return false;
  return true;
}
// The states and other plain arrays of a call must not overlap its sequence outputs.
inline bool clear_of(const void* p, size_t bytes, const Part* part, int n, size_t esz, bool written) {
  for (int i = 0; i < n; ++i)
    if ((part[i].out || written) && overlaps(p, bytes, part[i].p, (size_t)span(part[i].d, 0) * esz))
      return false;
  return true;
}

inline LaSeq in(const prnn_seq_t& x, int share) {
  return LaSeq{x.data, x.stride_t, x.stride_b, x.stride_h, share};
}

}  // namespace prnn
