// Host check of the barriers of the CTA-pair GEMM's ring of bits and scales: one
// copier that issues stages in order into a ring of slots, copies that land in any
// order, four groups that take every fourth stage, tensor cores that finish stages
// in order.  Random schedules; a group's wait may pass only once its stage's copy
// has landed, and its slot must not have been filled again.
#include <cstdio>
#include <random>
#include <vector>

#include "pair_ring.h"

using namespace mbok;

namespace {

// An mbarrier of one arrival per phase: completed phases.
struct Barrier {
  int phases = 0;
  // try_wait.parity: has the phase of this parity completed (the one before the current)?
  bool passes(unsigned parity) const { return (unsigned(phases) & 1u) != parity; }
};

bool run(int slots, int a_slots, unsigned seed) {
  std::mt19937 rng(seed);
  const int stages = 200;
  Barrier full[kPairMaxSlots], empty[kPairMaxSlots];
  std::vector<int> landed(stages, 0), unpacked(stages, 0);
  std::vector<int> in_flight, held(slots, -1);
  int issued = 0, done = 0;   // stages copied; stages whose products are complete
  int next[kPairGroups];
  bool past[kPairGroups] = {};   // the wait for its stage's bits has passed
  for (int g = 0; g < kPairGroups; ++g) next[g] = g;
  const int late = int(rng() % 8);   // how often a copy in flight is passed over
  for (int steps = 0; done < stages; ++steps) {
    if (steps > 1000000) {
      std::printf("slots %d, A slots %d, seed %u: stuck at stage %d\n", slots, a_slots, seed, done);
      return false;
    }
    switch (rng() % 4) {
      case 0: {   // the copier: once the slot's last stage is unpacked
        if (issued == stages) break;
        const int last = issued - slots;
        if (last >= 0 && !empty[pair_bits_barrier(last)].passes(pair_bits_parity(last))) break;
        if (last >= 0 && !unpacked[last]) {
          std::printf("slots %d, A slots %d, seed %u: stage %d filled over %d\n", slots, a_slots, seed, issued, last);
          return false;
        }
        held[issued % slots] = issued;
        in_flight.push_back(issued++);
        break;
      }
      case 1: {   // a copy lands, mostly not the oldest
        if (in_flight.empty()) break;
        size_t i = rng() % in_flight.size();
        if (i == 0 && int(rng() % 8) < late) break;
        const int g = in_flight[i];
        in_flight.erase(in_flight.begin() + long(i));
        landed[g] = 1;
        ++full[pair_bits_barrier(g)].phases;
        break;
      }
      case 2: {   // a group
        const int b = int(rng() % kPairGroups), g = next[b];
        if (g >= stages) break;
        // two waits, as in the kernel: for the bits, then for A's slot
        if (!past[b]) past[b] = full[pair_bits_barrier(g)].passes(pair_bits_parity(g));
        if (!past[b] || g >= done + a_slots) break;
        if (!landed[g] || held[g % slots] != g) {
          std::printf("slots %d, A slots %d, seed %u: the wait for stage %d passed before its copy\n", slots, a_slots,
                      seed, g);
          return false;
        }
        unpacked[g] = 1;
        ++empty[pair_bits_barrier(g)].phases;
        next[b] += kPairGroups;
        past[b] = false;
        break;
      }
      default:   // the tensor cores
        if (unpacked[done]) ++done;
    }
  }
  return true;
}

}  // namespace

int main() {
  int bad = 0;
  for (int slots = kPairGroups; slots <= kPairMaxSlots; ++slots)
    for (int a_slots = kPairGroups; a_slots <= kPairMaxSlots; ++a_slots)
      for (unsigned seed = 0; seed < 300; ++seed)
        if (!run(slots, a_slots, seed)) {
          ++bad;
          break;
        }
  return bad == 0 ? 0 : 1;
}
