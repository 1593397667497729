// w4_vector.hip -- the product with 4-bit weights for up to four rows of A: the codes' bytes
// bound it.
//
// Sixteen by sixteen blocks would be mostly empty, and turning codes into their operands costs
// more than the products: so here each lane keeps the 32 codes it loads (four lanes take 64
// consecutive bytes of a row, which the address unit takes in one cycle) and multiplies them with v_dot2, two
// products a lane.  WHOLE: groups are multiples of a step's 128 codes, one scale a step.  A lane's 32 codes lie in one group of scales in any case.  A's rows and
// the sums of their pieces of 32 come from LDS, the same for all 16 rows of W: a broadcast; they lie there in the
// order in which the codes are cheapest to turn (in_pairs()).
#include "w4_common.hpp"

namespace gemm {
namespace {

constexpr int kStep = 128;
constexpr int kSpan = 16384;   // elements of A in LDS at a time, all rows together

template <int T>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    if constexpr (T == DT_BF16) {
        typedef __bf16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
    }
}

struct Walk { int per, left, groups; };   // groups that WAVES steps cross, codes left over, all groups of a row

template <int T, int MR, int WAVES, bool WHOLE>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(4)))
void w4_vector_kernel(const W4Params p, const Walk walk) {
    constexpr int DEPTH = 4, SPAN = kSpan / MR;   // codes of a row per round of staging
    __shared__ __attribute__((aligned(16))) uint16_t held[MR * SPAN];
    __shared__ float sums[MR * SPAN / 32];
    __shared__ float part[WAVES][MR][16];
    const int lane = lane_id(), w = wave_id(), c = lane % 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, n = min(n0 + lane / 4, (int64_t)p.N - 1);
    const uint8_t* qsrc = p.W + n * p.ldw + 16 * c;
    const uint16_t* srow = reinterpret_cast<const uint16_t*>(p.scales) + n * p.lds;
    const uint16_t* zrow = reinterpret_cast<const uint16_t*>(p.zeros ? p.zeros : p.scales) + n * p.lds;   // (always loaded: no branch)
    const int full = p.K / kStep;
    const Spread<T> spread;
    u32x4 q[DEPTH];
    uint16_t sc[DEPTH], ze[DEPTH];
    float total[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) total[m] = 0.0f;

    // The group of the next step to load and the step's place in it, kept without divisions; a lane's
    // codes lie in that group or in one of the next three.
    int gi = w * kStep / p.group, in = w * kStep % p.group;
    auto load = [&](int d, int s) {   // steps are loaded in their order
        q[d] = load16(qsrc + (int64_t)s * (kStep / 2));
        int at = gi;
        if (!WHOLE) {
            const int k = in + 32 * c;
            at += (k >= p.group) + (k - p.group >= p.group) + (k - p.group - p.group >= p.group);
        }
        at = min(at, walk.groups - 1);
        sc[d] = srow[at];
        ze[d] = zrow[at];
        gi += walk.per;
        in += walk.left;
        if (in >= p.group) { in -= p.group; ++gi; }
    };
    auto multiply = [&](int k, const u32x4& word, float s, float z) {   // k: the step's place in LDS
        float dot[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) dot[m] = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            __builtin_amdgcn_sched_barrier(0);   // (the words mixed by the scheduler would not fit the registers)
            const u32x4 b = spread.in_pairs(word[t]);
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(held + m * SPAN + k + 32 * c + 8 * t);
#pragma unroll
                for (int e = 0; e < 4; ++e) dot[m] = dot2<T>(a[e], b[e], dot[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < MR; ++m)
            total[m] = __builtin_fmaf(s, __builtin_fmaf(-z, sums[(m * SPAN + k) / 32 + c], dot[m]), total[m]);
    };
    for (int64_t k0 = 0; k0 < p.K; k0 += SPAN) {
        const int s0 = (int)(k0 / kStep), s1 = (int)min((k0 + SPAN) / kStep, (int64_t)full);   // whole steps
        const int last = p.K - k0 < SPAN ? (int)((p.K - k0 + kStep - 1) / kStep) * kStep : SPAN;   // codes of this round, in steps
        auto piece = [&](int i) { return load_a(p.A + min(i / (SPAN / 8), p.M - 1) * p.lda * 2, (int)k0 + i % (SPAN / 8) * 8, p.K); };
        if (k0 > 0) { gi = ((int)k0 + w * kStep) / p.group; in = ((int)k0 + w * kStep) % p.group; }
        const u32x4 first = (int)threadIdx.x % (SPAN / 8) * 8 < last ? piece(threadIdx.x) : u32x4{0u, 0u, 0u, 0u};
        if (s1 > s0)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) load(d, min(s0 + w + d * WAVES, s1 - 1));
        if (k0 > 0) lds_barrier();   // every wave is done with the last round
#pragma unroll 1
        for (int i = threadIdx.x; i < MR * SPAN / 8; i += 64 * WAVES) {
            if (i % (SPAN / 8) * 8 >= last) continue;   // (whole groups of four threads: steps are 16 pieces)
            const u32x4 v = i == (int)threadIdx.x ? first : piece(i);
            *reinterpret_cast<u32x4*>(held + i * 8) = pairs_of(v);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += to_f32<T>((uint16_t)v[e]) + to_f32<T>((uint16_t)(v[e] >> 16));
            sum += __shfl_xor(sum, 1, 64);
            sum += __shfl_xor(sum, 2, 64);
            if (i % 4 == 0) sums[i / 4] = sum;
        }
        lds_barrier();
        // (loads stand outside of branches: behind one, a wait for an older load would wait for them all)
        for (int s = s0 + w; s < s1; s += DEPTH * WAVES)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (s + d * WAVES < s1)
                    multiply((s + d * WAVES - s0) * kStep, q[d], to_f32<T>(sc[d]), p.zeros ? zero16<T>(ze[d]) : kZero16);
                load(d, min(s + (d + DEPTH) * WAVES, s1 - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
        if (k0 + SPAN >= p.K && full * kStep < p.K && full % WAVES == w) {   // the last, partial step
            const int k = full * kStep + 32 * c;
            u32x4 word;
#pragma unroll
            for (int t = 0; t < 4; ++t) word[t] = load_q(qsrc - 16 * c, k + 8 * t, p.K);
            const int at = k < p.K ? k / p.group : 0;
            const float s = k < p.K ? to_f32<T>(srow[at]) : 0.0f, z = k >= p.K ? 0.0f : p.zeros ? zero16<T>(zrow[at]) : kZero16;
            multiply((int)(full * kStep - k0), word, s, z);
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        total[m] += __shfl_xor(total[m], 1, 64);
        total[m] += __shfl_xor(total[m], 2, 64);
        if (c == 0) part[w][m][lane / 4] = total[m];
    }
    lds_barrier();
    const int m = threadIdx.x / 16, col = threadIdx.x % 16;
    if (m >= MR || m >= p.M || n0 + col >= p.N) return;
    float v = 0.0f;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) v += part[x][m][col];
    store_c1(p.C, p.out_type, m * p.ldc + n0 + col, 16.0f * v, p.alpha, p.beta);
}

template <int T, int MR, int WAVES>
hipError_t go(const W4Params& p, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.N + 15) / 16)), block(64 * WAVES);
    const Walk walk = {WAVES * kStep / p.group, WAVES * kStep % p.group, (p.K + p.group - 1) / p.group};
    if (p.group % kStep == 0) hipLaunchKernelGGL((w4_vector_kernel<T, MR, WAVES, true>), grid, block, 0, st, p, walk);
    else hipLaunchKernelGGL((w4_vector_kernel<T, MR, WAVES, false>), grid, block, 0, st, p, walk);
    return hipGetLastError();
}
// Waves for 16 on each compute unit: what starts a wave (staging A, its addresses) costs as much as four
// steps, so no more than that share K.
template <int T, int MR>
hipError_t rows_of(const W4Params& p, hipStream_t st) {
    const int64_t blocks = ((int64_t)p.N + 15) / 16, cu = num_compute_units();
    if (blocks >= 3 * cu || p.K < 1024) return go<T, MR, 4>(p, st);
    return blocks >= 3 * cu / 2 || p.K < 4096 ? go<T, MR, 8>(p, st) : go<T, MR, 16>(p, st);
}
template <int T>
hipError_t vector_of(const W4Params& p, hipStream_t st) {
    return p.M == 1 ? rows_of<T, 1>(p, st) : p.M == 2 ? rows_of<T, 2>(p, st) : p.M <= 4 ? rows_of<T, 4>(p, st) : hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_w4_vector(int in_type, const W4Params& p, hipStream_t st) {
    return in_pieces(p, kW4VectorRows, kMostCols, [&](const W4Params& q) {
        return in_type == DT_BF16 ? vector_of<DT_BF16>(q, st) : vector_of<DT_F16>(q, st);
    });
}

}  // namespace gemm
