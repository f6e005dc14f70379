// Which tokens the rows of a chunk see (svq_tree_attention), a tile of 64 at a time: plain
// arithmetic on whole numbers, constexpr so that the host compiles what the kernels use.
#pragma once

#include <cstdint>

namespace svq {

constexpr int kTile = 64;   // tokens in a tile: bits of a mask
constexpr int kNodes = 64;  // trees up to this size have their paths as bits

// The lowest n bits, and all of them from n = 64 on.
constexpr uint64_t low_bits(int64_t n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Bit i at i + by; what leaves the 64 bits is gone. (Shifting by 64 or more is not that: the
// machine takes the amount modulo 64, and a path would come back in a tile far before it.)
constexpr uint64_t moved(uint64_t bits, int64_t by) {
    return by >= 64 || by <= -64 ? 0 : by >= 0 ? bits << by : bits >> -by;
}

// The cached tokens that a sequence's rows may see, numbered without gaps: the first ones
// (sinks) and then those from `from` on. The chunk's rows follow from number `cached` on.
struct Numbering {
    int len;     // cached tokens
    int sinks;   // tokens 0 .. sinks - 1 of the cache
    int from;
    int cached;  // how many there are

    constexpr void count(int window, int first) {
        sinks = 0;
        from = 0;
        if (window > 0) {
            sinks = first < 0 ? 0 : first < len ? first : len;
            // the first row, at position len, sees the window's oldest token
            from = len - window < 0 ? 0 : len - window + 1;
            if (from < sinks) from = sinks;
        }
        cached = sinks + len - from;
    }
    // place in the table of the cached token numbered u
    constexpr int position(int u) const { return u < sinks ? u : u - sinks + from; }
    // Tiles from this number on hold no token that only some of n rows are too deep to see: the
    // window's oldest token moves with the depth, and no row is deeper than n - 1.
    constexpr int edge(int window, int n) const { return window > 0 ? sinks + n - 1 : 0; }
    // Whether some row may not see some token of the tile from number `base` on, of which `there`
    // are there.
    constexpr bool needs_mask(int edge, int base, uint64_t there) const {
        return ~there != 0 || base + kTile > cached || (base < edge && base + kTile > sinks);
    }
    // The tokens that a row sees of the cache, of the tile from number `base` on.
    constexpr uint64_t cached_bits(int window, int base, int depth) const {
        uint64_t bits = low_bits((int64_t)cached - base);
        if (window > 0) {
            const int64_t past = (int64_t)len + depth - window + 1 - from;
            bits &= ~low_bits(sinks + (past > 0 ? past : 0) - base) | low_bits((int64_t)sinks - base);
        }
        return bits;
    }
    // Ancestors nearer than this are in the window; of depths below `sunk` all are first tokens.
    constexpr int far(int window) const { return window > 0 ? window : INT32_MAX; }
    constexpr int64_t sunk(int window, int first) const { return window > 0 ? (int64_t)first - len : 0; }

    // All that row `node` sees of a tile where every row's parent is the row before it; where
    // `line` holds a bit for each node of the row's path (trees of up to kNodes); where parents
    // are looked up (a negative one is none).
    constexpr uint64_t chain(int window, int first, int base, int node) const {
        const int64_t off = (int64_t)cached - base;  // bit of the sequence's first row
        const uint64_t line = low_bits(off + node + 1) & ~low_bits(off);
        const uint64_t kept = ~low_bits(off + (int64_t)node - far(window) + 1) | low_bits(off + sunk(window, first));
        return cached_bits(window, base, node) | (line & kept);
    }
    constexpr uint64_t path(int window, int first, int base, uint64_t line) const {
        // a path's nodes ascend with their depths
        const int depth = __builtin_popcountll(line) - 1;
        const int64_t sunk = this->sunk(window, first);
        uint64_t near = line, deep = line;
        for (int k = depth + 1 - far(window); k > 0; --k) near &= near - 1;
        for (int k = 0; k < sunk && deep; ++k) deep &= deep - 1;
        return cached_bits(window, base, depth) | moved(near | (line & ~deep), (int64_t)cached - base);
    }
    template <typename Parent>
    constexpr uint64_t walk(int window, int first, int base, int node, Parent parent_of) const {
        int depth = 0;  // (without a window it does not matter)
        if (window > 0)
            for (int i = parent_of(node); i >= 0; i = parent_of(i)) ++depth;
        const int64_t off = (int64_t)cached - base, sunk = this->sunk(window, first);
        uint64_t bits = cached_bits(window, base, depth);
        int d = 0;
        for (int i = node; i >= 0 && off + i >= 0; i = parent_of(i), ++d)
            if (off + i < 64 && (d < far(window) || depth - d < sunk)) bits |= 1ull << (off + i);
        return bits;
    }
};

}  // namespace svq
