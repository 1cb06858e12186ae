// Overlap check of the buffers a plan names (host only).
#pragma once
#include <stdint.h>

#include <algorithm>
#include <vector>

namespace qm {
namespace {

// Bytes [lo, hi) a buffer touches: all of them (pitch 0), or, for a strided
// grad, rows of `row` bytes every `pitch` bytes starting at lo.
struct Region {
    uintptr_t lo, hi, pitch, row;
};

// Whether two regions whose spans intersect share a byte.  Exact for two
// strided regions of one pitch (their rows occupy fixed column ranges modulo
// the pitch, e.g. column slices of one fused buffer); any other pair with
// intersecting spans counts as overlapping.
bool regions_overlap(const Region &x, const Region &y) {
    if (x.hi <= y.lo || y.hi <= x.lo) return false;
    if (!x.pitch || !y.pitch || x.pitch != y.pitch) return true;
    const uintptr_t P = x.pitch;
    const uintptr_t a = x.lo % P, b = y.lo % P;   // row starts modulo the pitch
    auto hits = [&](uintptr_t s0, uintptr_t l0, uintptr_t s1, uintptr_t l1) {
        // [s0, s0 + l0) and [s1, s1 + l1) on a circle of length P (l0, l1 <= P)
        const uintptr_t d = (s1 + P - s0) % P;
        return d < l0 || (P - d) % P < l1;
    };
    return hits(a, x.row, b, y.row);
}

// Whether any two of the regions share a byte (sorts them by address).
bool any_overlap(std::vector<Region> &spans) {
    std::sort(spans.begin(), spans.end(), [](const Region &x, const Region &y) { return x.lo < y.lo; });
    for (size_t k = 0; k < spans.size(); k++)
        for (size_t j = k + 1; j < spans.size() && spans[j].lo < spans[k].hi; j++)
            if (regions_overlap(spans[k], spans[j])) return true;
    return false;
}

}  // namespace
}  // namespace qm
