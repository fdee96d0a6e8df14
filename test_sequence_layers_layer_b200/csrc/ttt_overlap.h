// ttt_overlap.h -- the arrays of a call that may not share memory. Kernels of one call read
// some inputs again after they have written some outputs, in blocks that know nothing of one
// another, so an output that overlaps an input is an answer that is wrong without an
// error, but for the places where it may stand exactly over one.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ttt {

struct Range {
    const void *p;  // NULL: not there
    size_t n;       // bytes
};
struct OutRange {
    Range r;
    unsigned over;  // bit i: may be input i itself (the same address and size)
};

inline bool ranges_meet(const Range &a, const Range &b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y ? y - x < a.n : x - y < b.n;
}

// Whether an output meets another output, or an input that it may not stand over.
template <int NO, int NI>
bool outputs_clash(const OutRange (&out)[NO], const Range (&in)[NI]) {
    static_assert(NI <= 32, "a bit an input");
    for (int i = 0; i < NO; ++i) {
        const Range &o = out[i].r;
        for (int j = 0; j < i; ++j)
            if (ranges_meet(o, out[j].r)) return true;
        for (int j = 0; j < NI; ++j)
            if (ranges_meet(o, in[j]) &&
                !((out[i].over >> j & 1u) && o.p == in[j].p && o.n == in[j].n))
                return true;
    }
    return false;
}

}  // namespace ttt
