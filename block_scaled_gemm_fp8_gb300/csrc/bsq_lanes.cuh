// bsq_lanes.cuh -- lanes of a warp that hold the same number, shared by the router and the sort.
#pragma once

#include <cstdint>

namespace bsq {

constexpr uint32_t kFull = 0xffffffffu;

// The lanes whose v (below 2^bits) equals this lane's: a vote for each bit, four at a time (bits that all
// lanes lack change nothing).  A warp's match.any holds its SM quarter for 256 cycles on GB300 with 32
// different values (measured), a vote for 4.
__device__ __forceinline__ uint32_t same_lanes(uint32_t v, int bits) {
  uint32_t same = kFull;
  for (int b = 0; b < bits; b += 4, v >>= 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool set = v & (1u << i);
      const uint32_t votes = __ballot_sync(kFull, set);
      same &= set ? votes : ~votes;
    }
  }
  return same;
}

}  // namespace bsq
