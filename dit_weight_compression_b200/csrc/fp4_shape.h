// fp4_shape.h -- how many CTAs share one tile of a short 4-bit product.  Host code only, so that the rule can be
// checked without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace ep {
namespace fp4 {

constexpr int kMaxSplit = 8;

// CTAs of one tile: the most whose clusters all fit the device at once, with four stages each.  (4096
// outputs of 4096 for one token: 5.4 us with 4, 6.5 with 8 of two stages; 300 tokens: 11.1 us with 2, 16.7
// with 3, which need a second round.)  `clusters_of(split, n)` says how many clusters of `split` CTAs the
// device holds at once, and returns 0 or an error; none of a size (a part of a GPU may have no room for
// large clusters) means the next smaller one, down to CTAs by themselves.  An error, or no room for one
// CTA (`no_room`), is passed on.
template <class Error, class Query>
Error split_of(int64_t tiles, int steps, Query clusters_of, Error no_room, int& split) {
    for (split = std::min(kMaxSplit, (steps + 3) / 4);; --split) {
        int clusters = 0;
        const Error e = clusters_of(split, clusters);
        if (e != Error(0)) return e;
        if (split == 1) return clusters > 0 ? Error(0) : no_room;
        if (tiles <= clusters) return Error(0);
    }
}

}  // namespace fp4
}  // namespace ep
