// kv_tile_ring.h -- a loader's account of the tiles of a ring: how many it has taken, and
// which of their copies nobody else may be waiting for when the block gives up.  (No CUDA in
// it: tests run it on the CPU.)
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MK_RING __device__ __forceinline__
#else
#define MK_RING inline
#endif

namespace mk {

template <uint32_t NS>
struct TileRing {
  uint32_t tiles = 0;  // taken
  uint32_t whole = 0;  // by stage: whether the last tile there is one that this warp copies whole

  // Takes the next tile and says its stage.  waits: once free(stage, n) says that use n of the
  // stage, the one before, is over.  Where it does not, nothing is taken: the copy of that use
  // may be in flight, and stays among those that drain() waits for.
  template <class F>
  MK_RING bool take(bool waits, F free, uint32_t& stage) {
    stage = tiles % NS;
    if (waits && tiles >= NS && !free(stage, tiles / NS - 1)) return false;
    whole &= ~(1u << stage);
    tiles++;
    return true;
  }
  // The tile just taken is copied whole.
  MK_RING void copies(uint32_t stage) { whole |= 1u << stage; }
  // there(stage, n) for every stage whose last use, n, is a tile copied whole.
  template <class F>
  MK_RING void drain(F there) const {
    for (uint32_t i = tiles > NS ? tiles - NS : 0; i < tiles; i++)
      if (whole >> i % NS & 1) there(i % NS, i / NS);
  }
};

}  // namespace mk
