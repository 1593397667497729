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

template <int ACT, int T, int DT>
__device__ __forceinline__ void rows_of(const LinearBwdParams& p, int64_t m, int64_t end, int n, float (&sum)[8]) {
    constexpr int AHEAD = 4;
    for (; m < end; m += AHEAD * kLanes) {
        Eight<DT> dc[AHEAD];
        Eight<T> z[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int64_t r = m + a * kLanes;
            if (r >= end) continue;
            dc[a].load(p.dC + r * p.lddc * Elem<DT>::SIZE, n, 0, p.N);
            if constexpr (ACT != ACT_NONE) z[a].load(p.Z + r * p.ldz * 2, n, 0, p.N);
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int64_t r = m + a * kLanes;
            if (r >= end) continue;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = dc[a].get(i);
                if constexpr (ACT != ACT_NONE) v[i] *= slope_of<ACT>(z[a].get(i));
                sum[i] += v[i];
            }
            if (p.dZ) store8<T>(p.dZ + r * p.lddz * 2, n, 0, p.N, v);
        }
    }
}

template <int T, int DT>
__global__ __launch_bounds__(kCols / 8 * kLanes) void linear_bwd_kernel(const LinearBwdParams p) {
    constexpr int TPR = kCols / 8;
    __shared__ float sums[kLanes][kCols];
    const int c = (int)threadIdx.x % TPR, lane = (int)threadIdx.x / TPR;
    const int64_t col = (int64_t)blockIdx.x * kCols;
    const int n = (int)min(col + 8 * c, (int64_t)p.N);
    const int64_t per = (p.M + p.parts - 1) / p.parts, first = per * blockIdx.y, end = min(first + per, p.M);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n < p.N) {
        switch (p.act) {
            case ACT_NONE: rows_of<ACT_NONE, T, DT>(p, first + lane, end, n, sum); break;
            case ACT_RELU: rows_of<ACT_RELU, T, DT>(p, first + lane, end, n, sum); break;
            case ACT_GELU: rows_of<ACT_GELU, T, DT>(p, first + lane, end, n, sum); break;
            case ACT_GELU_TANH: rows_of<ACT_GELU_TANH, T, DT>(p, first + lane, end, n, sum); break;
            case ACT_SILU: rows_of<ACT_SILU, T, DT>(p, first + lane, end, n, sum); break;
        }
    }
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
        hipLaunchKernelGGL((linear_bwd_kernel<decltype(t)::value, decltype(d)::value>), grid, block, 0, st, p);
        return hipGetLastError();
    });
    if (e != hipSuccess || !p.db || p.parts == 1) return e;
    hipLaunchKernelGGL(linear_bwd_join_kernel, dim3((unsigned)((p.N + (int64_t)63) / 64)), dim3(256), 0, st, p.part, p.db, p.N, p.parts);
    return hipGetLastError();
}

}  // namespace gemm
