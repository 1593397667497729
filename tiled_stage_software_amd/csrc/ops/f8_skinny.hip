// f8_skinny.hip -- the 8-bit product for few rows of A: B's bytes bound it.
//
// A workgroup computes 16 columns (MT x 16 rows); its waves share K, each taking every
// kWaves-th step of 128 bytes.  Every lane loads its own 2 x 16 bytes of a row of B straight into
// registers as the matrix instruction's operand: nothing is read twice, so LDS would only add a
// trip.  kDepth steps are in flight per wave.  The waves' sums meet in LDS in wave order.
#include "f8_common.hpp"

namespace gemm {
namespace {

constexpr int kWaves = 8, kStep = 128;

template <int MT, bool WIDE>
__global__ __launch_bounds__(64 * kWaves) void f8_skinny_kernel(const F8Params p) {
    constexpr int DEPTH = MT == 1 ? 4 : 2;
    __shared__ float part[kWaves][MT][64][4];
    const int lane = lane_id(), w = wave_id(), r = lane % 16, g = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const uint8_t* brow = p.B + min(n0 + r, (int64_t)p.N - 1) * p.ldb;
    const uint8_t* arow[MT];
    bool has[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        has[i] = 16 * i + r < p.M;
        arow[i] = p.A + (int64_t)min(16 * i + r, p.M - 1) * p.lda;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 zero = {0u, 0u, 0u, 0u};
    // lane group g holds bytes 16 g and 64 + 16 g of a step: each load takes 64 whole bytes of 16 rows
    auto steps = [&](int s, auto count) {
        constexpr int D = decltype(count)::value;
        u32x4 b[D][2], a[D][MT][2];
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[d][h] = load16(brow + (int64_t)(s + d * kWaves) * kStep + 64 * h + 16 * g);
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    a[d][i][h] = zero;
                    if (has[i]) a[d][i][h] = load16(arow[i] + (int64_t)(s + d * kWaves) * kStep + 64 * h + 16 * g);
                }
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = mfma_f8<WIDE>(join16(b[d][0], b[d][1]), join16(a[d][i][0], a[d][i][1]), acc[i]);
    };
    const int full = p.K / kStep;
    int s = w;
    for (; s + (DEPTH - 1) * kWaves < full; s += DEPTH * kWaves) steps(s, std::integral_constant<int, DEPTH>());
    for (; s < full; s += kWaves) steps(s, std::integral_constant<int, 1>());
    if (s == full && full * kStep < p.K) {   // the last, partial step
        const int k = full * kStep + 16 * g;
        const i32x8 b = join16(load_chunk(brow, k, p.K), load_chunk(brow, k + 64, p.K));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            u32x4 lo = zero, hi = zero;
            if (has[i]) {
                lo = load_chunk(arow[i], k, p.K);
                hi = load_chunk(arow[i], k + 64, p.K);
            }
            acc[i] = mfma_f8<WIDE>(b, join16(lo, hi), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(part[w][i][lane]) = acc[i];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 256; t += 64 * kWaves) {
        const int n = t % 16, m = t / 16;
        if (m >= p.M || n0 + n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) v += part[q][m / 16][n / 4 * 16 + m % 16][n % 4];
        store_c1(p.C, p.out_type, m * p.ldc + n0 + n, v * (scale_or_one(p.sa, m) * scale_or_one(p.sb, n0 + n)), p.alpha, p.beta);
    }
}

template <int MT>
hipError_t go(const F8Params& p, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.N + 15) / 16)), block(64 * kWaves);
    if (p.out_type == DT_F32) hipLaunchKernelGGL((f8_skinny_kernel<MT, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((f8_skinny_kernel<MT, false>), grid, block, 0, st, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_skinny(const F8Params& p, hipStream_t st) {
    if (p.M <= 16) return go<1>(p, st);
    return p.M <= 32 ? go<2>(p, st) : hipErrorInvalidValue;
}

}  // namespace gemm
