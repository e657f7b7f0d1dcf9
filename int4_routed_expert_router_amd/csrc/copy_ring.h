// copy_ring.h -- the counted waits of a ring of three LDS stages.
//
// A wavefront's copies into LDS finish in the order they were issued, and a
// wait for n lets it pass once at most n of its vector-memory operations are
// in flight.  Plain C++, so that a host program can check the counts too.
#pragma once

namespace coli {

// Whether every stage has landed before the barrier behind which it is read.
// The prologue issues stage 0, two scale loads where there are scales, then
// stages 1 and 2, waits for `first` and reads stage 0; step st waits for
// `each`, passes the barrier, reads stage st + 1, and issues one scale load
// (with scales) and stage st + 3.  `copies` operations to a stage.
constexpr bool ring_waits_hold(int copies, bool scaled, int first, int each) {
  constexpr int kSteps = 12;
  int queue[(kSteps + 3) * 65 + 2] = {};  // stage of every operation; -1: a scale load
  int n = 0, done = 0;
  for (int i = 0; i < copies; ++i) queue[n++] = 0;
  for (int i = 0; i < (scaled ? 2 : 0); ++i) queue[n++] = -1;
  for (int i = 0; i < 2 * copies; ++i) queue[n++] = 1 + i / copies;
  if (n - first > done) done = n - first;
  for (int i = done; i < n; ++i)
    if (queue[i] == 0) return false;
  for (int st = 0; st < kSteps; ++st) {
    if (n - each > done) done = n - each;
    for (int i = done; i < n; ++i)
      if (queue[i] == st + 1) return false;
    if (scaled) queue[n++] = -1;
    for (int i = 0; i < copies; ++i) queue[n++] = st + 3;
  }
  return true;
}

}  // namespace coli
