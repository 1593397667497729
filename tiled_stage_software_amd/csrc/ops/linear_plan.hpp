// linear_plan.hpp -- which tiles and splits the products of gemm_linear and of its backward pass take.
#pragma once

#include <algorithm>

#include "ops.hpp"

namespace gemm {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct TilePlan {
    int bm, bn;    // rows and columns of a tile
    int splits;    // of the sum
};

// Where large tiles fill the card: the one with the least time on the fullest compute unit, a tile's elements, times kSmallCost where
// it is a small one.  Where small tiles do not fill it: the height and the splits of the sum that should be fastest.  A slab
// takes slab_us() on a compute unit that has nothing else to hide its loads with; more workgroups than units share them at kShared; a
// split writes and reads its fp32 sums once (at the rate of a copy) and needs one more launch.
constexpr double kSmallCost = 1.35, kShared = 0.75, kJoinUs = 4.0, kBytesPerUs = 4.5e6;
inline double slab_us(int bm) { return bm == 64 ? 0.35 : 0.5; }
inline double rounds_of(int64_t workgroups) {
    const int64_t cu = num_compute_units();
    return workgroups <= cu ? 1.0 : kShared * ceil_div(workgroups, cu);
}
// The best of the heights from `most` down to `least` (128 or 64) and of up to `splits` splits of `slabs`.
inline TilePlan small_plan(int64_t M, int64_t N, int64_t slabs, int most, int least, int64_t splits, int64_t ldp) {
    TilePlan q = {most, 128, 1};
    double best = 0.0;
    for (int bm = most; bm >= least; bm -= 64) {
        const int64_t tiles = ceil_div(M, bm) * ceil_div(N, 128);
        for (int64_t s = 1; s <= splits && s * 4 <= slabs + 3; ++s) {
            const double us = rounds_of(tiles * s) * ceil_div(slabs, s) * slab_us(bm) +
                              (s > 1 ? kJoinUs + s * (double)M * ldp * 8.0 / kBytesPerUs : 0.0);
            if (best == 0.0 || us < best) {
                best = us;
                q.bm = bm;
                q.splits = (int)s;
            }
        }
    }
    return q;
}

}  // namespace gemm
