// rows_pack.hpp -- operands' rows copied into a workspace for the products' direct loads: 16-byte aligned rows,
// a length that is whole slabs, as many rows as a tile, zeros for what is not there.
//
// The address unit takes four neighbouring lanes a cycle from aligned rows and about one from rows that start
// anywhere: 32 KiB of a slab then take a microsecond of a compute unit, twice what multiplying
// them does.  Copying costs each byte once; a tile of B is read by every row of tiles.
#pragma once

#include "f8_common.hpp"

namespace gemm {

constexpr int kRowsThreads = 256, kRowsEach = 4;   // 16-byte chunks per thread

// Block `block` of the copies of a (a_blocks of them) and b.
__device__ __forceinline__ void rows_pack(const RowsJob& a, const RowsJob& b, uint32_t a_blocks, uint32_t block) {
    const bool first = block < a_blocks;
    const RowsJob& j = first ? a : b;
    const uint32_t chunks = (uint32_t)(j.len_pad / 16), base = (first ? block : block - a_blocks) * (kRowsThreads * kRowsEach);
    u32x4 v[kRowsEach];
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const uint32_t id = base + i * kRowsThreads + threadIdx.x, row = id / chunks, k = (id - row * chunks) * 16;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (row < j.rows) v[i] = load_chunk(j.src + (int64_t)row * j.ld, (int)k, (int)j.len);
    }
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const uint32_t id = base + i * kRowsThreads + threadIdx.x;
        if (id < (uint32_t)j.rows_pad * chunks) *reinterpret_cast<u32x4*>(j.dst + (int64_t)id * 16) = v[i];
    }
}

inline uint32_t rows_pack_blocks(const RowsJob& j) {
    const int64_t chunks = (int64_t)j.rows_pad * (j.len_pad / 16);
    return j.src ? (uint32_t)((chunks + kRowsThreads * kRowsEach - 1) / (kRowsThreads * kRowsEach)) : 0;
}

}  // namespace gemm
