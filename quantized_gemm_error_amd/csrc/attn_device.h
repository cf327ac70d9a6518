// Device helpers shared by the attention kernels.
#pragma once

#include "attn_internal.h"
#include "device_common.h"

namespace spear {

// What the query at position p of a sequence of `len` cached tokens sees:
// positions [0, sink) and [lo, p], where sink <= lo; without a window sink is
// 0 and lo is 0.
struct Seen {
  int sink, lo;
};
__device__ __forceinline__ Seen seen_by(int p, int window, int sinks) {
  Seen s{0, 0};
  if (window > 0 && p >= window) {
    s.lo = p - window + 1;
    s.sink = min(sinks, s.lo);
  }
  return s;
}

// Cached tokens of sequence b, within what its table row can hold.
__device__ __forceinline__ int cached_len(const AttnDesc &d, int b) {
  return max(0, min(d.kv_lens[b], d.width * d.page_size));
}

}  // namespace spear
