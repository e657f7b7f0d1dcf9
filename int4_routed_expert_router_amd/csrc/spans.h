// spans.h -- ragged row spans (sequences, requests) on the device.
//
// n spans cover rows off[i] .. off[i+1] of a batch; off holds n + 1 ascending
// values, empty spans allowed.  Every lookup reads only off[0 .. n], also for
// a table that is not ascending, and every loop ends.
#pragma once

#include "device_common.h"

namespace coli {

// The last i in [0, n) with off[i] <= pos, or -1: a 64-way search, so tables
// of up to 64 entries take one load.  All 64 lanes take part.
COLI_DEV int last_at_or_before(const int32_t *__restrict__ off, int n, int pos) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;
  for (;;) {
    const int step = (len + 63) >> 6;
    const bool ok = lane * step < len && off[lo + lane * step] <= pos;
    const int cnt = __popcll(__ballot(ok));
    if (cnt == 0) return lo - 1 < 0 ? -1 : lo;
    lo += (cnt - 1) * step;
    if (step == 1) return lo;
    len = min(step, len - (cnt - 1) * step);
  }
}

// Requests and their adapters.  Rows in no request, and requests whose
// adapter is outside [0, n_adapters), have no adapter.
struct Requests {
  const int32_t *off;      // [n + 1]
  const int32_t *adapter;  // [n]
  int n, n_adapters;
};

// Calls f(ordinal, begin, end, adapter) for every request that has an adapter
// and rows in [lo, hi), in order, with begin and end clipped to that range.
// 64 requests are looked at per step.  All 64 lanes take part; the arguments
// of f are the same in all of them.
template <class F>
COLI_DEV void for_requests(const Requests &q, int lo, int hi, F f) {
  const int lane = threadIdx.x & 63;
  // up to 64 requests are one step anyway
  int s = q.n <= 64 ? 0 : max(0, last_at_or_before(q.off, q.n + 1, lo));
  int ordinal = 0;
  for (; s < q.n; s += 64) {
    const int i = min(s + lane, q.n - 1);
    const int b = q.off[i], e = q.off[i + 1], a = q.adapter[i];
    const int begin = max(b, lo), end = min(e, hi);
    const bool mine = s + lane < q.n && begin < end && a >= 0 && a < q.n_adapters;
    uint64_t todo = __ballot(mine);
    while (todo) {
      const int l = __ffsll((long long)todo) - 1;
      todo &= todo - 1;
      f(ordinal++, __builtin_amdgcn_readlane(begin, l), __builtin_amdgcn_readlane(end, l),
        __builtin_amdgcn_readlane(a, l));
    }
    if (__builtin_amdgcn_readlane(b, 63) >= hi) break;
  }
}

}  // namespace coli
