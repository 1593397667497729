// linear_bwd.hip -- what the backward pass of the product with bias, activation and residual does ahead of its two
// products:  dZ = dC * act'(Z),  db = sum over the rows of dZ.
//
// Bytes bound it.  A workgroup takes 256 columns of a run of rows: a thread keeps eight columns and every eighth row, so db is
// summed in registers, from unrounded values, and eight threads' sums meet in LDS.  Each run writes one row of
// partial sums, which a second launch adds in order; the same bits on every run.
#include <algorithm>

#include "linear.hpp"

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
        else dc[a].load(dc_at + r * dc_step, n, 0, p.N);
        if constexpr (ACT != ACT_NONE) {
            if constexpr (WHOLE) z[a].whole(z_at + r * z_step, n);
            else z[a].load(z_at + r * z_step, n, 0, p.N);
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
        }
    }
}

template <int T, int DT, int ACT>
__global__ __launch_bounds__(kCols / 8 * kLanes) void linear_bwd_kernel(const LinearBwdParams p) {
    constexpr int TPR = kCols / 8;
    __shared__ float sums[kLanes][kCols];
    const int c = (int)threadIdx.x % TPR, lane = (int)threadIdx.x / TPR;
    const int64_t col = (int64_t)blockIdx.x * kCols;
    const int n = (int)min(col + 8 * c, (int64_t)p.N);
    const int64_t per = (p.M + p.parts - 1) / p.parts, first = per * blockIdx.y, end = min(first + per, p.M);
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
        (p.parts > 1 ? p.part + (int64_t)blockIdx.y * p.N : p.db)[col + i] = s;
    }
}

// db = the parts' rows in order: 64 columns a workgroup, every fourth part a wave.
__global__ __launch_bounds__(256) void linear_bwd_join_kernel(const float* part, float* db, int N, int parts) {
    __shared__ float sums[4][64];
    const int64_t n = (int64_t)blockIdx.x * 64 + lane_id();
    const int w = wave_id();
    float s = 0.0f;
    if (n < N) {
#pragma unroll 8
        for (int i = w; i < parts; i += 4) s += part[(int64_t)i * N + n];
    }
    sums[w][lane_id()] = s;
    __syncthreads();
    if (w == 0 && n < N) db[n] = sums[0][lane_id()] + sums[1][lane_id()] + sums[2][lane_id()] + sums[3][lane_id()];
}

}  // namespace

// Runs of 32 rows at least (four rounds of a thread's loads), and no more than fill the card a few times over.
int linear_bwd_parts(int64_t M, int64_t N) {
    const int64_t strips = (N + kCols - 1) / kCols, most = 8 * (int64_t)num_compute_units();
    const int64_t want = std::max<int64_t>(1, most / std::max<int64_t>(1, strips)), rows = (M + 31) / 32;
    return (int)std::max<int64_t>(1, std::min(want, rows));
}

hipError_t launch_linear_bwd(int in_type, const LinearBwdParams& p, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + (int64_t)kCols - 1) / kCols), (unsigned)p.parts), block(kCols / 8 * kLanes);
    const hipError_t e = by_type(in_type, p.dc_type, [&](auto t, auto d) {
        auto go = [&](auto act) {
            hipLaunchKernelGGL((linear_bwd_kernel<decltype(t)::value, decltype(d)::value, decltype(act)::value>), grid, block, 0, st, p);
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
    if (e != hipSuccess || !p.db || p.parts == 1) return e;
    hipLaunchKernelGGL(linear_bwd_join_kernel, dim3((unsigned)((p.N + (int64_t)63) / 64)), dim3(256), 0, st, p.part, p.db, p.N, p.parts);
    return hipGetLastError();
}

}  // namespace gemm
