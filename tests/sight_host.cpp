// The masks of tree attention as the kernels compute them, for all tiles of one sequence.
#include <vector>

#include "svq_tree_sight.h"

using namespace svq;

// how: 0 a chain, 1 paths as bits, 2 parents looked up. Tiles begin at number `begin` and follow one
// another. masks [tiles][n], needs [tiles], positions of the first `cached` numbers; returns `cached`.
extern "C" int sight(int how, int n, const int32_t *parents, int len, int window, int first, int begin, int tiles,
                     uint64_t *masks, int32_t *needs, int32_t *positions) {
    Numbering t{};
    t.len = len;
    t.count(window, first);
    auto parent_of = [&](int i) { return parents[i] >= 0 && parents[i] < i ? parents[i] : -1; };
    std::vector<uint64_t> lines;
    for (int i = 0; how == 1 && i < n; ++i)
        lines.push_back(1ull << i | (parent_of(i) < 0 ? 0 : lines[parent_of(i)]));
    for (int k = 0; k < tiles; ++k) {
        const int base = begin + k * kTile;
        needs[k] = t.needs_mask(t.edge(window, n), base, ~0ull);
        for (int i = 0; i < n; ++i)
            masks[k * n + i] = how == 0   ? t.chain(window, first, base, i)
                               : how == 1 ? t.path(window, first, base, lines[i])
                                          : t.walk(window, first, base, i, parent_of);
    }
    for (int u = 0; u < t.cached; ++u) positions[u] = t.position(u);
    return t.cached;
}
