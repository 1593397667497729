// rows_pack.hip -- operands' rows copied into a workspace for the products' direct loads: 16-byte aligned rows,
// a length that is whole slabs, as many rows as a tile, zeros for what is not there.
//
// The address unit takes four neighbouring lanes a cycle from aligned rows and about one from rows that start
// anywhere: 32 KiB of a slab then take a microsecond of a compute unit, twice what multiplying
// them does.  Copying costs each byte once; a tile of B is read by every row of tiles.
#include "f8_common.hpp"

namespace gemm {
namespace {

constexpr int kThreads = 256, kEach = 4;   // 16-byte chunks per thread

__global__ __launch_bounds__(kThreads) void rows_pack_kernel(const RowsJob a, const RowsJob b, uint32_t a_blocks) {
    const bool first = blockIdx.x < a_blocks;
    const RowsJob& j = first ? a : b;
    const uint32_t chunks = (uint32_t)(j.len_pad / 16), base = (first ? blockIdx.x : blockIdx.x - a_blocks) * (kThreads * kEach);
    u32x4 v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t id = base + i * kThreads + threadIdx.x, row = id / chunks, k = (id - row * chunks) * 16;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (row < j.rows) v[i] = load_chunk(j.src + (int64_t)row * j.ld, (int)k, (int)j.len);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t id = base + i * kThreads + threadIdx.x;
        if (id < (uint32_t)j.rows_pad * chunks) *reinterpret_cast<u32x4*>(j.dst + (int64_t)id * 16) = v[i];
    }
}

uint32_t blocks_of(const RowsJob& j) {
    const int64_t chunks = (int64_t)j.rows_pad * (j.len_pad / 16);
    return j.src ? (uint32_t)((chunks + kThreads * kEach - 1) / (kThreads * kEach)) : 0;
}

}  // namespace

hipError_t launch_rows_pack(const RowsJob& a, const RowsJob& b, hipStream_t st) {
    const uint32_t na = blocks_of(a), nb = blocks_of(b);
    if (na + nb == 0) return hipSuccess;
    hipLaunchKernelGGL(rows_pack_kernel, dim3(na + nb), dim3(kThreads), 0, st, a, b, na);
    return hipGetLastError();
}

}  // namespace gemm
