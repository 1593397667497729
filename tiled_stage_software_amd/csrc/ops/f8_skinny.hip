// f8_skinny.hip -- the 8-bit product for few rows of A: B's bytes bound it.
//
// A workgroup computes 16 columns (MT x 16 rows); its waves share K, each taking every
// WAVES-th step of 128 bytes.  Every lane loads its own 2 x 16 bytes of a row of B straight into
// registers as the matrix instruction's operand: nothing is read twice, so LDS would only add a
// trip.  DEPTH steps are in flight per wave.  A last step that K does not fill is the row's last 128
// bytes, with zeros in A for what earlier steps had, so that it is in flight with the others.
// The waves' sums meet in LDS in wave order.
#include "f8_common.hpp"

namespace gemm {
namespace {

constexpr int kStep = 128;

template <int MT, int WAVES, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void f8_skinny_kernel(const F8Params p) {
    constexpr int DEPTH = MT == 1 ? 4 : 2;
    __shared__ float part[WAVES][MT][64][4];
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
    auto steps = [&](int s, auto last) {
        constexpr bool LAST = decltype(last)::value;
        u32x4 b[DEPTH][2], a[DEPTH][MT][2];
        int64_t k[DEPTH];
        int had[DEPTH];   // bytes of the step that earlier ones had (all of them past the last step)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            k[d] = (int64_t)(s + d * WAVES) * kStep;
            had[d] = 0;
            if (LAST && k[d] > p.K - kStep) {
                had[d] = (int)min(k[d] - (p.K - kStep), (int64_t)kStep);
                k[d] = p.K - kStep;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) b[d][h] = load16(brow + k[d] + 64 * h + 16 * g);
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    a[d][i][h] = zero;
                    if (has[i]) a[d][i][h] = load16(arow[i] + k[d] + 64 * h + 16 * g);
                }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (LAST && had[d] > 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int o = had[d] - (64 * h + 16 * g + 4 * q);
                        const uint32_t mask = o >= 4 ? 0u : o <= 0 ? ~0u : ~0u << (8 * o);
#pragma unroll
                        for (int i = 0; i < MT; ++i) a[d][i][h][q] &= mask;
                    }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = mfma_f8<WIDE>(join16(b[d][0], b[d][1]), join16(a[d][i][0], a[d][i][1]), acc[i]);
        }
    };
    if (p.K >= kStep) {
        const int count = (p.K + kStep - 1) / kStep;
        int s = w;
        for (; (s + (DEPTH - 1) * WAVES + 1) * (int64_t)kStep <= p.K; s += DEPTH * WAVES) steps(s, std::false_type());
        if (s < count) steps(s, std::true_type());
    } else if (w == 0) {
        const i32x8 b = join16(load_chunk(brow, 16 * g, p.K), load_chunk(brow, 64 + 16 * g, p.K));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            u32x4 lo = zero, hi = zero;
            if (has[i]) {
                lo = load_chunk(arow[i], 16 * g, p.K);
                hi = load_chunk(arow[i], 64 + 16 * g, p.K);
            }
            acc[i] = mfma_f8<WIDE>(b, join16(lo, hi), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(part[w][i][lane]) = acc[i];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 256; t += 64 * WAVES) {
        const int n = t % 16, m = t / 16;
        if (m >= p.M || n0 + n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) v += part[q][m / 16][n / 4 * 16 + m % 16][n % 4];
        store_c1(p.C, p.out_type, m * p.ldc + n0 + n, v * (scale_or_one(p.sa, m) * scale_or_one(p.sb, n0 + n)), p.alpha, p.beta);
    }
}

template <int MT, int WAVES>
hipError_t go(const F8Params& p, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.N + 15) / 16)), block(64 * WAVES);
    if (p.out_type == DT_F32) hipLaunchKernelGGL((f8_skinny_kernel<MT, WAVES, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((f8_skinny_kernel<MT, WAVES, false>), grid, block, 0, st, p);
    return hipGetLastError();
}

}  // namespace

// Sixteen waves where eight would leave most of the card's wave slots empty and each still has steps to take.
hipError_t launch_f8_skinny(const F8Params& p, hipStream_t st) {
    const bool deep = ((int64_t)p.N + 15) / 16 <= 2 * num_compute_units() && p.K >= 2048;
    if (p.M <= 16) return deep ? go<1, 16>(p, st) : go<1, 8>(p, st);
    if (p.M > kF8SkinnyRows) return hipErrorInvalidValue;
    return deep ? go<2, 16>(p, st) : go<2, 8>(p, st);
}

}  // namespace gemm
