// Rows of a ragged batch to their sequences.
#pragma once

#include <cstdint>

namespace mla {

// The last b in [0, B) with ro[b] <= t, for ro[0] <= t < ro[B]: a search in 32 parts
// by a whole warp.
__device__ __forceinline__ uint32_t find_sequence(const uint32_t* ro, uint32_t B, uint32_t t, int lane) {
  uint32_t lo = 0, hi = B;  // ro[lo] <= t < ro[hi]
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 31) / 32;
    const uint64_t at = lo + static_cast<uint64_t>(lane) * step;
    const bool below = at < hi && ro[at] <= t;
    const uint32_t votes = __ballot_sync(0xffffffffu, below);
    const uint32_t last = 31 - __clz(votes | 1u);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace mla
