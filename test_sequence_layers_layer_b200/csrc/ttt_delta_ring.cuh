// ttt_delta_ring.cuh -- rings of shared-memory stages that one thread keeps filled by bulk
// copies, for the scans of the gated delta rule. Uses mbar_wait() and mbar_drain() of the
// including source (sm100.cuh; a host test puts its own in their place).
#pragma once

#include <cstdint>

namespace ttt {
namespace delta {

constexpr int kScanStatus = 61;  // a wait of the scans has run out

// Place in a ring of stages: the stage and the parity of its use, without divisions.
struct Ring {
    int stages, s = 0, ph = 0;
    __device__ __forceinline__ explicit Ring(int n) : stages(n) {}
    __device__ __forceinline__ void next() {
        if (++s == stages) s = 0, ph ^= 1;
    }
};

// What one thread needs to keep a ring of stages filled. copy(step, stage, bar)
// issues the copies of a step after announcing their bytes on the barrier.
template <class Copy>
struct Filler {
    uint64_t *full, *empty;
    Copy copy;
    int steps, filled;
    Ring to;
    volatile int *abort;
    int *status;
    __device__ __forceinline__ Filler(uint64_t *f, uint64_t *e, int stages, int n, volatile int *ab,
                                      int *st, Copy c)
        : full(f), empty(e), copy(c), steps(n), filled(0), to(stages), abort(ab), status(st) {}
    // All steps, each waiting for its stage, up to the one whose wait runs out; then the
    // copies still in flight. This thread stays until they have landed, whoever gives up
    // meanwhile: an abort may be raised behind the last copy, and the block's shared memory
    // is not to go under it.
    __device__ __forceinline__ void run() {
        while (filled < steps) {
            if (filled >= to.stages && !mbar_wait(&empty[to.s], to.ph ^ 1, abort, status, kScanStatus))
                break;
            copy(filled, to.s, &full[to.s]);
            ++filled;
            to.next();
        }
        Ring r(to.stages);
        for (int i = 0; i < filled; ++i, r.next())
            if (i >= filled - to.stages) mbar_drain(&full[r.s], r.ph);
    }
};

}  // namespace delta
}  // namespace ttt
