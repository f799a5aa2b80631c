// The length of the pieces that a batch of cached sequences is cut into, for the
// kernel of gdr_cache.hip; plain arithmetic, the same on the host.
#pragma once

#include <math.h>
#include <stdint.h>

namespace gdr {

constexpr int kMaxPieces = 256;  // of one sequence
constexpr uint32_t kLeast = 64;  // keys of a piece at least

// Keys of a piece, whole tiles: an even share for each of `slots`, `sum` keys in all,
// the longest sequence `most` (at most 2^30) of them.  A share may be many times the
// longest sequence, where there are fewer slots than sequences, and past 32 bits: no
// piece needs more than that sequence.
__host__ __device__ inline uint32_t piece_keys(double sum, uint32_t most, int slots, uint32_t tile) {
  const double even = ceil(sum / static_cast<double>(slots));
  uint32_t per = even < static_cast<double>(most) ? static_cast<uint32_t>(even) : most;
  const uint32_t few = (most + kMaxPieces - 1) / kMaxPieces;
  per = per < few ? few : per;
  per = per < kLeast ? kLeast : per;
  return (per + tile - 1) / tile * tile;
}

}  // namespace gdr
