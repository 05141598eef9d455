// A loading warp's way around a ring of tiles in shared memory (host code too, so that its counts are tested without a GPU).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DSA_RING_FN __host__ __device__ __forceinline__
#else
#define DSA_RING_FN inline
#endif

namespace dsa {

// Tile i of a sequence lies in place i % kRing; kStep warps bring them, warp w the tiles w, w + kStep, w + 2 kStep, ...
template <uint32_t kRing, uint32_t kStep>
struct TileRing {
  static_assert(kStep >= 1 && kStep <= kRing, "a step stays within two rounds");
  uint32_t at;          // place of the warp's next tile
  uint32_t round = 0;   // how often that was used before
  uint32_t issued = 0;  // its tiles whose copies were issued

  DSA_RING_FN explicit TileRing(uint32_t warp) : at(warp) {}

  // The next tile's copies are issued.
  DSA_RING_FN void next() {
    ++issued;
    at += kStep;
    if (at >= kRing) {
      at -= kRing;
      ++round;
    }
  }
};

// f(place, parity) of the barriers behind which copies may be in flight once every warp has issued its last, `issued` of them each,
// wherever in a block it gave up: those of the last tile in each place (one before it has landed, or the place were not taken again).
template <uint32_t kRing, uint32_t kStep, class Counts, class F>
DSA_RING_FN void tiles_in_flight(const Counts& issued, F f) {
  uint32_t end = 0;  // behind the last tile
  for (uint32_t w = 0; w < kStep; ++w) {
    const uint32_t n = issued[w];
    if (n > 0 && w + kStep * (n - 1) + 1 > end) end = w + kStep * (n - 1) + 1;
  }
  for (uint32_t place = 0; place < kRing && place < end; ++place) {
    uint32_t tile = end - 1 - (end - 1 - place) % kRing;
    while (tile >= kRing && tile / kStep >= issued[tile % kStep]) tile -= kRing;
    if (tile / kStep < issued[tile % kStep]) f(place, tile / kRing & 1u);
  }
}

}  // namespace dsa
