// The refusal of overlapping arrays (ttt_overlap.h), for CPU tests. TEST CODE ONLY.
#include "../../test_sequence_layers_layer_b200/csrc/ttt_overlap.h"

// Two outputs (the first may stand over input 1) and three inputs: address, bytes each.
extern "C" int overlap_host_run(const unsigned long long *a) {
    auto at = [&](int i) { return ttt::Range{reinterpret_cast<const void *>(a[2 * i]), (size_t)a[2 * i + 1]}; };
    const ttt::OutRange out[] = {{at(0), 1u << 1}, {at(1), 0}};
    const ttt::Range in[] = {at(2), at(3), at(4)};
    return ttt::outputs_clash(out, in);
}
