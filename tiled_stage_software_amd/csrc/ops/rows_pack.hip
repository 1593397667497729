// rows_pack.hip -- the copies of rows_pack.hpp as a launch of their own.
#include "rows_pack.hpp"

namespace gemm {
namespace {

__global__ __launch_bounds__(kRowsThreads) void rows_pack_kernel(const RowsJob a, const RowsJob b, uint32_t a_blocks) {
    rows_pack(a, b, a_blocks, blockIdx.x);
}

}  // namespace

hipError_t launch_rows_pack(const RowsJob& a, const RowsJob& b, hipStream_t st) {
    const uint32_t na = rows_pack_blocks(a), nb = rows_pack_blocks(b);
    if (na + nb == 0) return hipSuccess;
    hipLaunchKernelGGL(rows_pack_kernel, dim3(na + nb), dim3(kRowsThreads), 0, st, a, b, na);
    return hipGetLastError();
}

}  // namespace gemm
