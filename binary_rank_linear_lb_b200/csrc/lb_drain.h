// Where a draining warp of a persistent CTA is in its tiles.  Two accumulators take turns:
// the CTA's tile number i is in accumulator i & 1, and its sums are there when that
// accumulator's "full" barrier has completed phase i / 2.
// (In a file of its own, without CUDA, so that it also runs on the host.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define LB_DRAIN __device__ __forceinline__
#else
#define LB_DRAIN inline
#endif

namespace lb {

// For each tile: full(wait) once, store the tile (its sums, or NaN where full was false),
// give the accumulator back if alive, next().
//
// Giving up is for good.  A barrier that no phase is completed on any more answers the
// wait for the phase after with yes (of a phase only the parity is asked for), so every
// other tile behind the lost one would pass for summed.  Nor is an accumulator given
// back any more: another warp may still be reading the sums that it waited for.
struct DrainTurn {
    int i = 0;
    bool alive = true;

    LB_DRAIN uint32_t buf() const { return (uint32_t)i & 1u; }
    // wait(parity): waits for that phase of buf()'s barrier; false: it gave up.
    template <class Wait>
    LB_DRAIN bool full(Wait wait) {
        alive = alive && wait((uint32_t)(i >> 1) & 1u);
        return alive;
    }
    LB_DRAIN void next() { ++i; }
};

}  // namespace lb
