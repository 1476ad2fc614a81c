// The waits of a ring of stages that gives up, against a model of its barriers:
// whatever has landed, the waits all succeed exactly when nothing is in flight.
#include <cstdio>
#include <vector>

#include "rr_turns.h"

// A barrier that has completed `phases` phases: a wait for a parity succeeds if
// the current, incomplete phase is of the other one.
static bool done(unsigned phases, unsigned parity) { return (phases & 1) != parity; }

int main() {
  unsigned long cases = 0;
  for (unsigned S = 1; S <= 6; ++S)
    for (unsigned end = 0; end <= 5 * S; ++end) {
      const unsigned first = end > S ? end - S : 0, open = end - first;
      for (unsigned landed = 0; landed < (1u << open); ++landed) {
        // turn q was issued after turn q - S was over, so a stage's last turn is
        // the only one that may be in flight
        std::vector<unsigned> phases(S, 0);
        for (unsigned q = 0; q < end; ++q)
          if (q < first || (landed >> (q - first) & 1)) ++phases[q % S];
        unsigned waits = 0;
        bool all = true;
        std::vector<bool> seen(S, false);
        rr::each_open_turn(end, S, [&](unsigned stage, unsigned parity) {
          ++waits;
          if (stage >= S || seen[stage]) all = false, waits = ~0u / 2;
          seen[stage % S] = true;
          all = all && done(phases[stage], parity);
        });
        if (waits != open || all != (landed == (1u << open) - 1)) {
          std::printf("stages %u, turns %u, landed %x: %u waits, %s\n", S, end, landed, waits, all ? "all" : "not all");
          return 1;
        }
        ++cases;
      }
    }
  std::printf("ok %lu\n", cases);
  return 0;
}
