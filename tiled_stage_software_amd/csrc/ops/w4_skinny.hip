// w4_skinny.hip -- C = alpha * A * W^T + beta * C with 4-bit weights for few rows of A: the
// codes' bytes bound it.
//
// A workgroup computes 16 columns; its waves share K, each taking every WAVES-th step of 128
// codes.  Every lane loads 16 bytes (32 codes) of a row of W straight into registers: the four
// lane groups take 64 whole bytes of a row.  An instruction's k have to lie in one group of
// scales, which may be 32 long, so the four words of a lane change places with those of the other lane
// groups (a 4 x 4 transpose, four lane swaps) until instruction t holds k = 32 t .. 32 t + 31.
// The sum of a, which the zero points multiply, is one more instruction, against ones.
#include "w4_common.hpp"

namespace gemm {
namespace {

constexpr int kStep = 128;

// v[i] of lane group g becomes v[g] of lane group i.
__device__ __forceinline__ u32x4 transpose_groups(u32x4 v) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    const u2 a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const u2 b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    const u2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const u2 d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// MT x 16 rows.  CHAIN: instructions of 32 codes that are sure to share a scale (groups are multiples of 32 * CHAIN).
template <int T, int MT, int WAVES, int CHAIN>
__global__ __launch_bounds__(64 * WAVES) void w4_skinny_kernel(const W4Params p, int tiles_n) {
    constexpr int NS = 4 / CHAIN, DEPTH = MT == 1 && (WAVES == 8 || NS < 4) ? 4 : 2;   // (what the registers hold)
    __shared__ float part[WAVES][MT][64][4];
    const int lane = lane_id(), w = wave_id(), r = lane % 16, g = lane / 16;
    const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * 16;
    const int m0 = (int)(blockIdx.x / tiles_n) * 16 * MT;
    const int64_t nc = min(n0 + r, (int64_t)p.N - 1);
    const uint8_t* qrow = p.W + nc * p.ldw;
    const uint16_t* srow = reinterpret_cast<const uint16_t*>(p.scales) + nc * p.lds;
    const uint16_t* zrow = reinterpret_cast<const uint16_t*>(p.zeros) + nc * p.lds;
    const char* arow[MT];
    bool has[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        has[i] = m0 + 16 * i + r < p.M;
        arow[i] = p.A + (int64_t)min(m0 + 16 * i + r, p.M - 1) * p.lda * 2;
    }
    const u32x4 none = {0u, 0u, 0u, 0u}, ones = {Half<T>::ONES, Half<T>::ONES, Half<T>::ONES, Half<T>::ONES};
    f32x4 total[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) total[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // 128 codes: words q of this lane in instruction order, a[i][t] the matching elements of A, and NS scales
    auto multiply = [&](const u32x4& q, const u32x4 (*a)[4], const float* s, const float* z) {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        f32x4 dot[MT], sum[MT];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const u32x4 b = spread<T>(q[t]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const bool first = t % CHAIN == 0;
                dot[i] = Half<T>::mfma(a[i][t], b, first ? zero : dot[i]);
                sum[i] = Half<T>::mfma(a[i][t], ones, first ? zero : sum[i]);
                if (t % CHAIN == CHAIN - 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[i][e] = __builtin_fmaf(s[t / CHAIN], __builtin_fmaf(-z[t / CHAIN], sum[i][e], dot[i][e]), total[i][e]);
                }
            }
        }
    };
    const int full = p.K / kStep;
    // D steps from s, every WAVES-th.  LAST: those past the last whole step repeat it with zeros in A and scales.
    auto steps = [&](int s, auto depth, auto last) {
        constexpr int D = decltype(depth)::value;
        constexpr bool LAST = decltype(last)::value;
        u32x4 q[D], a[D][MT][4];
        uint16_t sb[D][NS], zb[D][NS];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int st = LAST ? min(s + d * WAVES, full - 1) : s + d * WAVES;
            q[d] = load16(qrow + (int64_t)st * (kStep / 2) + 16 * g);
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int64_t gi = (st * kStep + 32 * CHAIN * j) / p.group;
                sb[d][j] = srow[gi];
                zb[d][j] = p.zeros ? zrow[gi] : (uint16_t)0;
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const bool in = !LAST || s + d * WAVES < full;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    a[d][i][t] = none;
                    if (has[i] && in) a[d][i][t] = load16(arow[i] + ((int64_t)(s + d * WAVES) * kStep + 32 * t + 8 * g) * 2);
                }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            float sc[NS], ze[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                sc[j] = !LAST || s + d * WAVES < full ? scale16<T>(sb[d][j]) : 0.0f;
                ze[j] = p.zeros ? zero16<T>(zb[d][j]) : kZero16;
                if (LAST && s + d * WAVES >= full) ze[j] = 0.0f;
            }
            multiply(transpose_groups(q[d]), a[d], sc, ze);
        }
    };
    int s = w;
    for (; s + (DEPTH - 1) * WAVES < full; s += DEPTH * WAVES)
        steps(s, std::integral_constant<int, DEPTH>(), std::false_type());
    if (s < full) steps(s, std::integral_constant<int, DEPTH>(), std::true_type());
    if (full % WAVES == w && full * kStep < p.K) {   // the last, partial step
        u32x4 q, a[MT][4];
        float sc[NS], ze[NS];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int k = full * kStep + 32 * t + 8 * g;
            q[t] = load_q(qrow, k, p.K);
#pragma unroll
            for (int i = 0; i < MT; ++i) a[i][t] = has[i] ? load_a(arow[i], k, p.K) : none;
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int64_t k = full * kStep + 32 * CHAIN * j;
            const bool in = k < p.K;
            sc[j] = in ? scale16<T>(srow[k / p.group]) : 0.0f;
            ze[j] = !in ? 0.0f : p.zeros ? zero16<T>(zrow[k / p.group]) : kZero16;
        }
        multiply(q, a, sc, ze);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(part[w][i][lane]) = total[i];
    __syncthreads();
    // lane l, element e holds row 4 * (l / 16) + e and column l % 16; the waves' sums meet in wave order
    for (int t = threadIdx.x; t < MT * 256; t += 64 * WAVES) {
        const int n = t % 16, row = t / 16, m = m0 + row;
        if (m >= p.M || n0 + n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) v += part[q][row / 16][row % 16 / 4 * 16 + n][row % 4];
        store_c1(p.C, p.out_type, m * p.ldc + n0 + n, v, p.alpha, p.beta);
    }
}

template <int T, int MT, int WAVES>
hipError_t go(const W4Params& p, hipStream_t st) {
    const int64_t tn = ((int64_t)p.N + 15) / 16, tm = ((int64_t)p.M + 16 * MT - 1) / (16 * MT);
    if (tm * tn > INT32_MAX / (64 * WAVES)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(tm * tn)), block(64 * WAVES);
    if (p.group % 128 == 0) hipLaunchKernelGGL((w4_skinny_kernel<T, MT, WAVES, 4>), grid, block, 0, st, p, (int)tn);
    else if (p.group % 64 == 0) hipLaunchKernelGGL((w4_skinny_kernel<T, MT, WAVES, 2>), grid, block, 0, st, p, (int)tn);
    else hipLaunchKernelGGL((w4_skinny_kernel<T, MT, WAVES, 1>), grid, block, 0, st, p, (int)tn);
    return hipGetLastError();
}

// Sixteen waves where eight would leave most of the card's wave slots empty and each still has steps to take.
template <int T>
hipError_t skinny_of(const W4Params& p, hipStream_t st) {
    const int64_t tn = ((int64_t)p.N + 15) / 16;
    const bool deep = tn <= 2 * num_compute_units() && p.K >= 2048;
    if (p.M <= 16) return deep ? go<T, 1, 16>(p, st) : go<T, 1, 8>(p, st);
    return go<T, 4, 8>(p, st);
}

}  // namespace

hipError_t launch_w4_skinny(int in_type, const W4Params& p, hipStream_t st) {
    return in_type == DT_BF16 ? skinny_of<DT_BF16>(p, st) : skinny_of<DT_F16>(p, st);
}

}  // namespace gemm
