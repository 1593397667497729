// w4_skinny.hip -- C = alpha * A * W^T + beta * C with 4-bit weights for few rows of A: the
// codes' bytes bound it.
//
// A workgroup computes 16 columns (MT x 16 rows); its waves share K, each taking every WAVES-th
// step of 128 codes, DEPTH steps of loads ahead of the one it multiplies.
//
// The address unit takes four neighbouring lanes a cycle only if they lie in one cache line, so
// no load follows the matrix instruction's layout (lane l holds row l % 16): four lanes load 64
// consecutive bytes of codes of a row, sixteen lanes 256 bytes of A, and a slot of LDS that belongs to the
// wave turns them (no barrier: a wave's LDS operations run in order).  Instruction t of a step
// takes k = 32 t .. 32 t + 31, which one group of scales holds.  The scales and zero points of the 16
// columns are brought into LDS by the whole workgroup before it starts: gathered step by step
// they took as many cycles of the address unit as all the rest (16 rows of A, groups of 64: 33 us of
// 4096 x 14336, of which the codes' bytes take 7).
#include "w4_common.hpp"

namespace gemm {
namespace {

constexpr int kStep = 128;
constexpr int64_t kMostRows = int64_t(1) << 20;   // of a launch: blocks of 32 rows are its grid's second size

// CHAIN: instructions of 32 codes that are sure to share a scale (groups are multiples of 32 * CHAIN).
template <int T, int MT, int WAVES, int CHAIN>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(MT == 1 ? 4 : 2)))
void w4_skinny_kernel(const W4Params p) {
    constexpr int DEPTH = 2;   // what the registers of four (MT 1) or two waves a SIMD hold
    constexpr int AL = 4 * MT;                 // 16-byte loads of A per step, four rows each
    constexpr int QB = 16 * 64, SLOT = QB + AL * 4 * 256;
    constexpr int NG = WAVES == 16 ? 256 : 128;          // groups of each column in LDS at a time
    constexpr int GROW = NG + 1;                         // apart: columns start on different banks
    constexpr int GROUPS = 16 * GROW * 8;              // of each the scale and 1 + z/16 as floats
    __shared__ __attribute__((aligned(1024))) char smem_raw[WAVES * (SLOT > MT * 1024 ? SLOT : MT * 1024) + GROUPS];
    LDS_AS char* slot = (LDS_AS char*)smem_raw + wave_id() * SLOT;
    LDS_AS f32x2* groups = reinterpret_cast<LDS_AS f32x2*>((LDS_AS char*)smem_raw + sizeof(smem_raw) - GROUPS);
    const int lane = lane_id(), w = wave_id(), r = lane % 16, g = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int m0 = (int)blockIdx.y * 16 * MT;
    const uint8_t* qsrc = p.W + min(n0 + lane / 4, (int64_t)p.N - 1) * p.ldw + 16 * (lane % 4);
    const char* asrc[AL];
#pragma unroll
    for (int h = 0; h < AL; ++h) asrc[h] = p.A + ((int64_t)min(m0 + g + 4 * h, p.M - 1) * p.lda + 8 * r) * 2;   // rows past the end are not stored
    const u32x4 ones = {Half<T>::ONES, Half<T>::ONES, Half<T>::ONES, Half<T>::ONES};
    const Spread<T> spread;
    f32x4 total[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) total[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 q[DEPTH], a[DEPTH][AL];

    const int full = p.K / kStep;
    auto load = [&](int d, int s) {
        q[d] = load16(qsrc + (int64_t)s * (kStep / 2));
#pragma unroll
        for (int h = 0; h < AL; ++h) a[d][h] = load16(asrc[h] + (int64_t)s * (kStep * 2));
    };
    // Chunk c of A's row `row` of the slot: 16 lanes of one chunk and 16 rows meet 16 different ones.
    auto a_at = [&](int row, int c) { return reinterpret_cast<LDS_AS u32x4*>(slot + QB + row * 256 + ((c ^ (row & 15)) << 4)); };
    // at: the first instruction's group in LDS; in: k's place in it; left: codes before the end (past it A is
    // zero and a group need not exist).
    auto multiply = [&](int at, int in, int left, const uint32_t* word, auto&& chunk) {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        f32x4 dot[MT], sum[MT];
        f32x2 sz = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const bool first = t % CHAIN == 0, last = t % CHAIN == CHAIN - 1;
            if (first) {
                sz = groups[r * GROW + at];
                if (left <= 32 * t) sz = f32x2{0.f, 0.f};
                in += 32 * CHAIN;
                if (in >= p.group && left > 32 * (t + CHAIN)) { in = 0; ++at; }
            }
            const u32x4 b = spread.in_order(word[t]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const u32x4 f = chunk(i, t);
                dot[i] = Half<T>::mfma(f, b, first ? zero : dot[i]);
                sum[i] = Half<T>::mfma(f, ones, first ? zero : sum[i]);
                if (last) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        total[i][e] = __builtin_fmaf(sz[0], __builtin_fmaf(-sz[1], sum[i][e], dot[i][e]), total[i][e]);
                }
            }
        }
    };
    auto step = [&](int d, int at, int in, int left) {
        wave_fence();
        const int row = lane / 4;
        *reinterpret_cast<LDS_AS u32x4*>(slot + row * 64 + (((lane % 4) ^ swz<4>(row)) << 4)) = q[d];
#pragma unroll
        for (int h = 0; h < AL; ++h) *a_at(g + 4 * h, r) = a[d][h];
        wave_fence();
        uint32_t word[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) word[t] = *reinterpret_cast<LDS_AS uint32_t*>(slot + r * 64 + ((t ^ swz<4>(r)) << 4) + 4 * g);
        multiply(at, in, left, word, [&](int i, int t) -> u32x4 {
            return *a_at(16 * i + r, 4 * t + g);
        });
        __builtin_amdgcn_sched_barrier(0);   // steps mixed by the scheduler would not fit the registers
    };
    // Groups that LDS holds at a time are whole steps; their steps are dealt to the waves.
    const int64_t span = (int64_t)p.group * NG;   // codes (a multiple of 128)
    for (int64_t k0 = 0; k0 < p.K; k0 += span) {
        const int s0 = (int)(k0 / kStep), s1 = (int)min((k0 + span) / kStep, (int64_t)full);   // whole steps
        if (s1 > s0)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) load(d, min(s0 + w + d * WAVES, s1 - 1));
        if (k0 > 0) lds_barrier();   // every wave is done with the last groups
        const int g0 = (int)(k0 / p.group);
        const int ng = min(NG, (p.K + p.group - 1) / p.group - g0);
        const int row = threadIdx.x / (4 * WAVES);
        for (int c = threadIdx.x % (4 * WAVES); c < ng; c += 4 * WAVES) {
            const int64_t at = min(n0 + row, (int64_t)p.N - 1) * p.lds + g0 + c;
            groups[row * GROW + c] = f32x2{to_f32<T>(reinterpret_cast<const uint16_t*>(p.scales)[at]),
                                                p.zeros ? zero16<T>(reinterpret_cast<const uint16_t*>(p.zeros)[at]) : kZero16};
        }
        lds_barrier();
        // (loads stand outside of branches: behind one, a wait for an older load would wait for them all)
        int at = w * kStep / p.group, in = w * kStep % p.group;   // this step's first group, and its place in it
        for (int s = s0 + w; s < s1; s += DEPTH * WAVES)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (s + d * WAVES < s1) step(d, at, in, kStep);
                load(d, min(s + (d + DEPTH) * WAVES, s1 - 1));
                at += WAVES * kStep / p.group;
                in += WAVES * kStep % p.group;
                if (in >= p.group) { in -= p.group; ++at; }
            }
        if (k0 + span >= p.K && full * kStep < p.K && full % WAVES == w) {   // the last, partial step
            const int k = full * kStep, at = k / p.group;
            q[0] = load_q16(p.W + min(n0 + lane / 4, (int64_t)p.N - 1) * p.ldw, k + 32 * (lane % 4), p.K);
#pragma unroll
            for (int h = 0; h < AL; ++h) a[0][h] = load_a(p.A + (int64_t)min(m0 + g + 4 * h, p.M - 1) * p.lda * 2, k + 8 * r, p.K);
            step(0, at - g0, k - at * p.group, p.K - k);
        }
    }
    lds_barrier();   // the slots are free
    auto part = [&](int v, int i, int l) { return reinterpret_cast<LDS_AS f32x4*>((LDS_AS char*)smem_raw + ((v * MT + i) * 64 + l) * 16); };
#pragma unroll
    for (int i = 0; i < MT; ++i) *part(w, i, lane) = total[i];
    lds_barrier();
    // lane l, element e holds row 4 * (l / 16) + e and column l % 16; the waves' sums meet in wave order
    for (int t = threadIdx.x; t < MT * 256; t += 64 * WAVES) {
        const int n = t % 16, m = t / 16;
        if (m0 + m >= p.M || n0 + n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int x = 0; x < WAVES; ++x) v += reinterpret_cast<LDS_AS float*>(part(x, m / 16, m % 16 / 4 * 16 + n))[m % 4];
        store_c1(p.C, p.out_type, (m0 + m) * p.ldc + n0 + n, 16.0f * v, p.alpha, p.beta);
    }
}

template <int T, int MT, int WAVES>
hipError_t go(const W4Params& p, hipStream_t st) {
    const int64_t tn = ((int64_t)p.N + 15) / 16, tm = ((int64_t)p.M + 16 * MT - 1) / (16 * MT);
    const dim3 grid((unsigned)tn, (unsigned)tm), block(64 * WAVES);
    if (p.group % 128 == 0) hipLaunchKernelGGL((w4_skinny_kernel<T, MT, WAVES, 4>), grid, block, 0, st, p);
    else if (p.group % 64 == 0) hipLaunchKernelGGL((w4_skinny_kernel<T, MT, WAVES, 2>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((w4_skinny_kernel<T, MT, WAVES, 1>), grid, block, 0, st, p);
    return hipGetLastError();
}

// Waves for 16 on each compute unit (a wave's start costs as much as some steps, so no more share K).
int w4_waves(const W4Params& p, int mt) {
    const int64_t blocks = ((int64_t)p.N + 15) / 16 * ((p.M + 16 * mt - 1) / (16 * mt)), cu = num_compute_units();
    if (blocks >= 3 * cu || p.K < 1024) return 4;
    return mt > 1 || blocks >= 3 * cu / 2 || p.K < 4096 ? 8 : 16;
}
template <int T, int MT>
hipError_t rows_of(const W4Params& p, hipStream_t st) {
    const int waves = w4_waves(p, MT);
    if (waves == 4) return go<T, MT, 4>(p, st);
    return waves == 8 ? go<T, MT, 8>(p, st) : go<T, 1, 16>(p, st);
}
template <int T>
hipError_t skinny_of(const W4Params& p, hipStream_t st) {
    return p.M <= 16 ? rows_of<T, 1>(p, st) : rows_of<T, 2>(p, st);
}

}  // namespace

// Expected microseconds: rounds of workgroups, each a start and its waves' steps in turn (measured from 1 to 32 steps
// and 1 to 112 rounds).  Groups below 128 end more often; rows that are not 16-byte aligned take two lines a load
// (128 x 3001 x 9001, groups of 64: 70 us, on tiles with copied rows 39).
double w4_skinny_us(const W4Params& p) {
    const int64_t mt = p.M <= 16 ? 1 : 2, blocks = ((int64_t)p.N + 15) / 16 * ((p.M + 16 * mt - 1) / (16 * mt));
    const int64_t waves = w4_waves(p, (int)mt), at_once = num_compute_units() * (mt == 1 ? 16 : 8) / waves;
    const double steps = (double)(((int64_t)p.K + kStep * waves - 1) / (kStep * waves));
    const bool aligned = ((uintptr_t)p.A | (uintptr_t)p.W | (uint64_t)p.lda * 2 | (uint64_t)p.ldw) % 16 == 0;
    const double step_us = 0.95 * (p.group < 128 ? 1.2 : 1.0) * (aligned ? 1.0 : 2.0);
    return 3.0 + (double)((blocks + at_once - 1) / at_once) * (2.7 + step_us * steps);
}

hipError_t launch_w4_skinny(int in_type, const W4Params& p, hipStream_t st) {
    return in_pieces(p, kMostRows, kMostCols, [&](const W4Params& q) {
        return in_type == DT_BF16 ? skinny_of<DT_BF16>(q, st) : skinny_of<DT_F16>(q, st);
    });
}

}  // namespace gemm
