// linear_attention_plan.h -- how the time axis of linear attention is cut, for the
// tensor-core and the CUDA-core kernels alike.
#pragma once

#include <algorithm>
#include <cstddef>

#include "seq_internal.h"

namespace prnn {

// A CTA walks the chunks of one (role, sequence, head, slice of columns) one after another.  With few of
// those the time axis is cut into `segs` runs of cps chunks that go side by side; the states that enter
// them come from a first pass over b and c, which leaves the state of every run of cpb chunks (cps is a
// multiple of cpb) in the scratch, `subs` of them.
struct LaPlan {
  int segs, cps, subs, cpb, slices;
};

// places: CTAs that run at once.  The estimate counts chunk times of one CTA: a chunk of the first
// pass costs about `first` of one, a CTA's start one, the second launch three.  The first pass's states fit
// `capacity` bytes at state_bytes each.
inline LaPlan la_plan(const LaArgs& a, int chunk, int slice, int places, double first,
                      size_t state_bytes, size_t capacity) {
  LaPlan p{1, 1, 0, 1, 1};
  bool in_place = false;  // a segment could write the state before another has read it
  int e = 0;
  for (int i = 0; i < a.roles; ++i) {
    in_place = in_place || (a.role[i].x0 && a.role[i].x0 == a.role[i].x_end);
    e = std::max(e, a.role[i].e);
  }
  const int chunks = (a.T + chunk - 1) / chunk;
  p.slices = (e + slice - 1) / slice;
  p.cps = chunks;
  const long long ctas = (long long)a.B * a.H * p.slices * a.roles;
  auto waves = [&](long long n) { return (double)((n + places - 1) / places); };
  double best = waves(ctas) * (chunks + 1);
  if (in_place) return p;
  for (int want = 2; want <= 64 && want <= chunks; ++want)
    for (int m = 1; m <= 4; ++m) {
      const int cpb = (chunks + want * m - 1) / (want * m), cps = cpb * m;
      const int segs = (chunks + cps - 1) / cps, subs = (segs - 1) * m;
      if (segs < 2 || (size_t)ctas * subs * state_bytes > capacity) continue;
      const double cost = waves(ctas * segs) * (cps + 1) + waves(ctas * subs) * (first * cpb + 1) +
                          3 + 0.05 * subs;
      if (cost < best) {
        best = cost;
        p = {segs, cps, subs, cpb, p.slices};
      }
    }
  return p;
}

}  // namespace prnn
