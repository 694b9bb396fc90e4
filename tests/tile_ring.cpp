// A loader's account of its tiles (csrc/kv_tile_ring.h) against a model of the copies in
// flight: give-ups at every step, over all orders of whole and made tiles of some length.
#include <cstdio>
#include <vector>

#include "kv_tile_ring.h"

template <uint32_t NS>
static long check(int steps) {
  long bad = 0;
  for (uint32_t kinds = 0; kinds < 1u << steps; kinds++)
    for (int last = 0; last <= steps; last++) {  // the step whose wait gives up (steps: none)
      mk::TileRing<NS> ring;
      std::vector<long> in_flight(NS, -1);  // by stage: the tile whose copy may not have landed
      uint32_t taken = 0;
      for (int i = 0; i < steps; i++) {
        uint32_t stage = ~0u;
        const bool got = ring.take(
            true,
            [&](uint32_t s, uint32_t use) {
              if (s != taken % NS || use != taken / NS - 1) bad++;  // the use before, of the next stage
              if (i >= last) return false;
              in_flight[s] = -1;  // used, so landed
              return true;
            },
            stage);
        if (!got) break;
        if (stage != taken % NS || in_flight[stage] >= 0) bad++;
        if (kinds >> i & 1) {
          ring.copies(stage);
          in_flight[stage] = taken;
        }
        taken++;
      }
      ring.drain([&](uint32_t s, uint32_t use) {
        if (in_flight[s] != (long)(use * NS + s)) bad++;  // a phase that does not come, or is past
        in_flight[s] = -1;
      });
      for (long tile : in_flight) bad += tile >= 0;
    }
  return bad;
}

int main() {
  const long bad = check<2>(9) + check<4>(13);
  printf("%ld\n", bad);
  return bad != 0;
}
