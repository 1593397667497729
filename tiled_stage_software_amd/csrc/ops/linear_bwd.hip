// linear_bwd.hip -- what the backward pass of the product with bias, activation and residual does ahead of its two
// products:  dZ = dC * act'(Z),  db = sum over the rows of dZ.
//
// Bytes bound it (4096 x 14336 bf16 with gelu: 74 us, 4.8 TB/s).  A workgroup takes 256 columns of a run of rows: a thread keeps eight
// columns and every eighth row, so db is summed in registers, from unrounded values, and eight threads' sums meet in LDS.  Each run
// writes one row of partial sums, which the launch that ends the backward pass adds in order; the same bits on every run.  Where the
// products need aligned rows, dZ is written a second time in such rows, and the other operands' copies ride in the same launch.
//
// dZ is rounded to the operands' 16 bits, the pass's one rounding beside its results': the matrix instructions take both operands in
// that type, and a dZ in two parts would double both products.  It is what bf16 gradients are off by: 0.0023 of their size (0.0017 is
// the result's own rounding), 0.0017 where dW is fp32; f16 an eighth of that.  From the products of the dZ that is stored, an fp32
// dW is 1e-7 off, and db, of unrounded values, from the formula.
#include <algorithm>

#include "linear.hpp"
#include "rows_pack.hpp"

namespace gemm {
namespace {

constexpr int kCols = 256, kLanes = 8;   // columns of a workgroup, rows at a time

// Rows m, m + kLanes, ... below `end` of columns n .. n+7.  WHOLE: all eight are there, and nothing stands behind a branch: the
// next rows' loads run under this row's operations and stores.
template <int ACT, int T, int DT, bool WHOLE>
__device__ __forceinline__ void rows_of(const LinearBwdParams& p, int64_t m, int64_t end, int n, float (&sum)[8]) {
    constexpr int AHEAD = 2;
    const int64_t dc_step = p.lddc * Elem<DT>::SIZE * kLanes, z_step = p.ldz * 2 * kLanes, dz_step = p.lddz * 2 * kLanes;
    const char* dc_at = p.dC + m * p.lddc * Elem<DT>::SIZE;
    const char* z_at = p.Z + m * p.ldz * 2;
    char* dz_at = p.dZ + m * p.lddz * 2;
    const int64_t rows = m < end ? (end - m + kLanes - 1) / kLanes : 0;   // this thread's
    Eight<DT> dc[AHEAD];
    Eight<T> z[AHEAD];
    auto load = [&](int a, int64_t i) {   // (past the last row: the last again)
        const int64_t r = i < rows ? i : rows - 1;
        if constexpr (WHOLE) dc[a].whole(dc_at + r * dc_step, n);
        else dc[a].load(dc_at + r * dc_step, n, p.N);
        if constexpr (ACT != ACT_NONE) {
            if constexpr (WHOLE) z[a].whole(z_at + r * z_step, n);
            else z[a].load(z_at + r * z_step, n, p.N);
        }
    };
    if (rows == 0) return;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) load(a, a);
    for (int64_t i = 0; i < rows; i += AHEAD) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = dc[a].get(e);
            if constexpr (ACT != ACT_NONE) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= slope_of<ACT>(z[a].get(e));
            }
            load(a, i + a + AHEAD);
            if (i + a >= rows) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += v[e];
            if (p.dZ) store8<T>(dz_at + (i + a) * dz_step, n, 0, p.N, v);
            if (p.copy) store16(p.copy + ((m + (i + a) * kLanes) * p.ldcopy + n) * 2, Elem<T>::pack(v));   // (zeros past N)
        }
    }
}

template <int T, int DT, int ACT>
__global__ __launch_bounds__(kCols / 8 * kLanes) void linear_bwd_kernel(const LinearBwdParams p, uint32_t blocks, uint32_t strips, uint32_t a_blocks) {
    constexpr int TPR = kCols / 8;
    static_assert(kCols / 8 * kLanes == kRowsThreads, "the copies' workgroups are these");
    if (blockIdx.x >= blocks) {
        rows_pack(p.jobs[0], p.jobs[1], a_blocks, blockIdx.x - blocks);
        return;
    }
    const uint32_t strip = blockIdx.x % strips, part = blockIdx.x / strips;
    __shared__ float sums[kLanes][kCols];
    const int c = (int)threadIdx.x % TPR, lane = (int)threadIdx.x / TPR;
    const int64_t col = (int64_t)strip * kCols;
    const int n = (int)min(col + 8 * c, (int64_t)p.N);
    const int64_t per = (p.M + p.parts - 1) / p.parts, first = per * part, end = min(first + per, p.M);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col + kCols <= p.N) rows_of<ACT, T, DT, true>(p, first + lane, end, n, sum);   // the same for the workgroup
    else if (n < p.N) rows_of<ACT, T, DT, false>(p, first + lane, end, n, sum);
    if (!p.db) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[lane][8 * c + i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kCols; i += TPR * kLanes) {
        if (col + i >= p.N) break;
        float s = 0.0f;
#pragma unroll
        for (int l = 0; l < kLanes; ++l) s += sums[l][i];
        (p.parts > 1 ? p.part + (int64_t)part * p.N : p.db)[col + i] = s;
    }
}

}  // namespace

// Runs of 32 rows at least (four rounds of a thread's loads), of half as many while that leaves compute units empty, and no more than fill
// the card a few times over.
int linear_bwd_parts(int64_t M, int64_t N) {
    const int64_t strips = std::max<int64_t>(1, (N + kCols - 1) / kCols), cu = num_compute_units();
    int64_t run = 32;
    while (run > kLanes && strips * ((M + run / 2 - 1) / (run / 2)) <= cu * 3 / 4) run /= 2;
    return (int)std::max<int64_t>(1, std::min(8 * cu / strips, (M + run - 1) / run));
}

hipError_t launch_linear_bwd(int in_type, const LinearBwdParams& p, hipStream_t st) {
    const uint32_t strips = (uint32_t)((p.N + (int64_t)kCols - 1) / kCols), blocks = strips * (uint32_t)p.parts;
    const uint32_t a_blocks = rows_pack_blocks(p.jobs[0]), grid = blocks + a_blocks + rows_pack_blocks(p.jobs[1]);
    return by_type(in_type, p.dc_type, [&](auto t, auto d) {
        auto go = [&](auto act) {
            hipLaunchKernelGGL((linear_bwd_kernel<decltype(t)::value, decltype(d)::value, decltype(act)::value>), dim3(grid),
                               dim3(kCols / 8 * kLanes), 0, st, p, blocks, strips, a_blocks);
            return hipGetLastError();
        };
        switch (p.act) {
            case ACT_RELU: return go(std::integral_constant<int, ACT_RELU>{});
            case ACT_GELU: return go(std::integral_constant<int, ACT_GELU>{});
            case ACT_GELU_TANH: return go(std::integral_constant<int, ACT_GELU_TANH>{});
            case ACT_SILU: return go(std::integral_constant<int, ACT_SILU>{});
        }
        return go(std::integral_constant<int, ACT_NONE>{});
    });
}

}  // namespace gemm
