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

// What tiles should take, in microseconds beside what all have in common (333 x 3001 x 2049 to 128 x 1593 x 8799, tiles of 64 and 128 rows,
// 1 to 8 splits): a slab on a compute unit that has nothing else to hide its loads with, and how much longer from rows of any
// alignment; more workgroups than units share them at kShared; a split writes and reads its fp32 sums once and needs one more
// launch, as copies of rows do, which find part of them in the caches.  A large tile's elements against a small one's: kSmallCost.
constexpr double kSmallCost = 1.35, kShared = 0.75, kJoinUs = 3.0, kBytesPerUs = 4.5e6, kCopyUs = 3.5, kCopiedPerUs = 6.5e6;
inline double slab_us(int bm) { return bm == 64 ? 0.26 : 0.39; }
inline double staged_us(int bm) { return bm == 64 ? 0.24 : 0.28; }
inline double rounds_of(int64_t workgroups) {
    const int64_t cu = num_compute_units();
    return workgroups <= cu ? 1.0 : kShared * ceil_div(workgroups, cu);
}

}  // namespace gemm
