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

// What tiles should take, in microseconds beside what all have in common.  Measured: a slab of 64 of K on the fullest compute unit, from
// the tiles that come to it (1 to 10 a unit on 512 x 7680 x 4096 to 1024 x 20480 x 4096).  One alone has the ring of four slots; of
// more, two run at a time, each hiding the other's waits.  LOADS: direct, or through registers from rows of any alignment.
// A split writes and reads its fp32 sums once and needs one more launch, as copies of rows do, which find part of them in the caches.
enum : int { DIRECT = 0, STAGED = 1 };
constexpr double kJoinUs = 3.0, kBytesPerUs = 4.5e6, kCopyUs = 3.5, kCopiedPerUs = 5.5e6;
inline double slabs_us(int64_t cu, int bm, int64_t workgroups, int64_t slabs, int loads) {
    const int64_t n = (workgroups + cu - 1) / cu;
    if (bm > 128) return n * slabs * (bm == 256 ? 1.57 : 1.26);
    const bool low = bm == 64, staged = loads == STAGED;
    const double alone = low ? (staged ? 0.52 : 0.32) : staged ? 0.66 : 0.45;
    const double one = low ? (staged ? 0.52 : 0.37) : staged ? 0.66 : 0.68, two = low ? (staged ? 1.0 : 0.6) : staged ? 1.46 : 0.9;
    return slabs * (n == 1 ? alone : n / 2 * two + n % 2 * one);
}

constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 12, 16, 24, 32, 48, 64};   // that are tried

}  // namespace gemm
