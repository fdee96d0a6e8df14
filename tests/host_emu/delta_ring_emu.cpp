// Host run of the thread that keeps a ring of stages filled (ttt_delta_ring.cuh) on a
// simulated ring: a copy lands, and a consumer gives a stage back, only when the model's
// clock has gone on, which a wait does. TEST CODE ONLY.
#include <cstdint>
#include <vector>

#undef __device__
#undef __forceinline__
#define __device__
#define __forceinline__ inline

namespace {
constexpr int kMaxStages = 8;
struct Sim {
    int stages, give_up;             // give_up: the consumer stops after so many steps (-1: never)
    long clock = 0;
    long lands[kMaxStages];          // when the copy of a stage's current use lands
    int use[kMaxStages];             // uses of a stage so far
    int consumed = 0;                // steps that the consumer has given back
    bool aborted = false, misuse = false;
    std::vector<int> steps;
    // the consumer takes a landed step, in order, a tick after it landed
    void tick() {
        ++clock;
        if (give_up >= 0 && consumed >= give_up) {
            aborted = true;
            return;
        }
        if (consumed < (int)steps.size() && lands[consumed % stages] < clock) ++consumed;
    }
} sim;
uint64_t full_[kMaxStages], empty_[kMaxStages];
}  // namespace

namespace ttt {
namespace delta {
// Stage s has been given back for the use'th time once the consumer has passed its step.
inline bool mbar_wait(uint64_t *bar, int parity, volatile int *, int *status, int code) {
    const int s = (int)(bar - empty_);
    const int use = sim.use[s] - 1;  // the use to be given back
    if (use < 0 || (use & 1) != parity) sim.misuse = true;
    for (int i = 0; i < 1000; ++i) {
        if (sim.consumed > use * sim.stages + s) return true;
        if (sim.aborted) return false;
        sim.tick();
    }
    *status = code;
    return false;
}
inline bool mbar_drain(uint64_t *bar, int parity) {
    const int s = (int)(bar - full_);
    if (sim.use[s] < 1 || ((sim.use[s] - 1) & 1) != parity) sim.misuse = true;
    while (sim.clock < sim.lands[s]) sim.tick();
    return true;
}
}  // namespace delta
}  // namespace ttt

#include "../../test_sequence_layers_layer_b200/csrc/ttt_delta_ring.cuh"

// Copies in flight when the filling thread is gone, or -1 (barriers misused), -2 (a stage
// overwritten before it was given back), -3 (steps out of order); *done: steps issued.
extern "C" int delta_ring_host_run(int stages, int steps, int latency, int give_up, int *done) {
    sim = Sim{};
    sim.stages = stages, sim.give_up = give_up;
    for (int s = 0; s < kMaxStages; ++s) sim.lands[s] = 0, sim.use[s] = 0;
    bool early = false, order = true;
    auto copy = [&](int step, int s, uint64_t *bar) {
        if (bar != full_ + s || s != step % stages) order = false;
        if (step >= stages && sim.consumed <= step - stages) early = true;
        sim.lands[s] = sim.clock + latency;
        ++sim.use[s];
        sim.steps.push_back(step);
    };
    int abort = 0, status = 0;
    ttt::delta::Filler<decltype(copy)> f(full_, empty_, stages, steps, &abort, &status, copy);
    f.run();
    *done = (int)sim.steps.size();
    if (sim.misuse) return -1;
    if (early) return -2;
    for (int i = 0; i < *done; ++i) order = order && sim.steps[i] == i;
    if (!order) return -3;
    int flying = 0;
    for (int s = 0; s < stages && s < *done; ++s) flying += sim.lands[s] > sim.clock;
    return flying;
}
