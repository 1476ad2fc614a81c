// rr_turns.h -- the turns of a ring of shared-memory stages, in plain C++ (also
// compiled for the host by the tests).
#pragma once

#ifdef __CUDACC__
#define RR_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RR_HOST_DEVICE inline
#endif

namespace rr {

// Turn q of a ring of S stages takes stage q % S, and a barrier of that stage
// completes one phase a turn: turn q's is the one of this parity.
RR_HOST_DEVICE constexpr unsigned turn_parity(unsigned q, unsigned S) { return (q / S) & 1; }

// wait(stage, parity) for each turn before `end` whose stage no later one has
// taken: those may still be in flight when no more are issued (turn q was
// issued only after turn q - S was over).
template <class F>
RR_HOST_DEVICE void each_open_turn(unsigned end, unsigned S, F wait) {
  for (unsigned q = end > S ? end - S : 0; q < end; ++q) wait(q % S, turn_parity(q, S));
}

}  // namespace rr
