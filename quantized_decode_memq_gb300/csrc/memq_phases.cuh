// memq_phases.cuh -- which phases of its barriers a producer of TMA copies has announced.  Plain C++, so
// that a test on the host runs the same arithmetic.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MEMQ_HD __host__ __device__ __forceinline__
#else
#define MEMQ_HD inline
#endif

namespace memq {

// Counts grow only where bytes are announced on a barrier, so that what is in flight can be awaited
// whenever the producer stops: use number n of a barrier (from 0) completes its phase n.
struct CopyPhases {
    uint32_t slot = 0, lap = 0;        // ring slot of the next piece, uses of that slot so far
    uint32_t scales = 0, ropes = 0;    // tiles whose scales, whose position parts were announced

    MEMQ_HD void piece_announced(uint32_t slots) {
        if (++slot == slots) {
            slot = 0;
            ++lap;
        }
    }
    // Uses so far of ring slot s, of scale buffer b (tiles alternate between two).
    MEMQ_HD uint32_t pieces_in(uint32_t s) const { return lap + (s < slot ? 1 : 0); }
    MEMQ_HD uint32_t scales_in(uint32_t b) const { return (scales + 1 - b) >> 1; }
};

// Parity to wait for until use number `uses - 1` of a barrier is complete.
MEMQ_HD uint32_t last_parity(uint32_t uses) { return (uses - 1) & 1; }

}  // namespace memq
