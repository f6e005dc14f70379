// What the C entry points look at in their arguments (host code that runs before any HIP call).
#pragma once

#include <cstddef>
#include <cstdint>

namespace svq {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    const void *p;
    size_t bytes;
};

inline bool overlap(const Span &a, const Span &b) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return pa < pb + b.bytes && pb < pa + a.bytes;
}

// Whether any of `outs` overlaps another of them or any of `ins` (null entries are skipped).
inline bool any_overlap(const Span *outs, int no, const Span *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        if (!outs[i].p) continue;
        for (int j = i + 1; j < no; ++j)
            if (outs[j].p && overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < ni; ++j)
            if (ins[j].p && overlap(outs[i], ins[j])) return true;
    }
    return false;
}

// Whether na columns from `a` on and nb columns from `b` on, of a matrix of 2-byte elements with
// row stride ld that holds both, share none (both are 2-byte aligned). Their rows alternate in memory.
inline bool columns_apart(const void *a, int64_t na, const void *b, int64_t nb, int64_t ld) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    if (pb < pa) return columns_apart(b, nb, a, na, ld);
    const int64_t q = (int64_t)((pb - pa) / 2 % (uintptr_t)ld);
    return q >= na && q + nb <= ld;
}

}  // namespace svq
