// clip_rules.h -- how a clipping goes by the size of its plan.
#pragma once

#include <cstdint>

namespace coli {

// A plan's bytes are judged item by item: by an item's own times the items
// there are.  Exact for one gradient up to its last item; of a plan of unequal
// items the full ones overrate it and the short ones underrate it.  The bytes of
// an item from which that comes to `bytes`:
constexpr int clip_item_from(int64_t bytes, int64_t n_items) {
  const int64_t from = (bytes + n_items - 1) / n_items;
  return from < 0x7fffffff ? (int)from : 0x7fffffff;
}
constexpr int clip_item_bytes(int32_t n, bool f32) { return n << (f32 ? 2 : 1); }

// From a quarter of the chip's last cache on the sum reads past it: 656 MB in
// 95 us instead of 141, 110 MB in 18 instead of 29.  Below, what writes the
// results gains more by finding there what the sum has read (both, into other
// buffers: 16 MB 11.8 us, past it 13.0; 32 MB 18.5 and 20.2, in bf16 18.4 and
// 20.2; 64 MB 38.6 and 38.4).
constexpr int64_t kSumPast = int64_t(64) << 20;

// Results that would not stay in the last cache anyway are read and written
// past it (656 MB: 222 us instead of 233; all of 256 MB 269 instead of 280 with
// an update from them behind; 128 MB 138 against 137, in bf16 140 against 136,
// 20,000 gradients of 1,000 values 98 against 96).
constexpr int64_t kScalePast = int64_t(256) << 20;

// The partial sums are added up once, in a launch between the two, where that
// takes less than every workgroup of the second adding them up itself, which
// is one to an item: 4,096 items of 256 values 10.2 us instead of 11.5, 5,000
// of 300 12.3 instead of 14.1, 20,000 of 64 23 instead of 34, 656 MB in place
// without clipping 109 instead of 121; 2,048 items 12.2 against 11.8, 3,000 of
// 8,000 values 57.4 against 56.3.
constexpr int64_t kSumOnce = 4096;

}  // namespace coli
