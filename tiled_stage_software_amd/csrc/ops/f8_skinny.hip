// f8_skinny.hip -- the 8-bit product for few rows of A: B's bytes bound it.
//
// A workgroup computes 16 columns (MT x 16 rows); its waves share K, each taking every
// WAVES-th step of 128 bytes, DEPTH steps of loads ahead of the one it multiplies.
//
// The matrix instruction wants lane l to hold row l % 16, but the address unit takes four
// neighbouring lanes a cycle only if they lie in one cache line: loaded as the instruction wants
// them, a row's 16 bytes to a lane, a KiB took 64 cycles of it, which bound the kernel at 16 bytes per cycle
// and compute unit.  So eight lanes load 128 consecutive bytes of a row (16 cycles a KiB), and a
// slot of LDS that belongs to the wave turns them: no barrier, the wave's LDS operations run in
// order.  A goes the same way; FEW: at most kFewRows rows, a quarter of the loads.
//
// A last step that K does not fill is the row's last 128 bytes, with zeros in A for what earlier
// steps had.  The waves' sums meet in LDS in wave order.
#include "f8_common.hpp"

namespace gemm {
namespace {

constexpr int kStep = 128, kFewRows = 4;

template <int MT, int WAVES, bool WIDE, bool FEW>
__global__ __launch_bounds__(64 * WAVES) void f8_skinny_kernel(const F8Params p) {
    constexpr int DEPTH = MT == 1 || WAVES == 8 ? 4 : 2;   // what the registers hold
    constexpr int AL = FEW ? 1 : 2 * MT;                  // 16-byte loads of A per step, eight rows each
    constexpr int SLOT = (16 + 8 * AL) * kStep;
    static_assert(!FEW || MT == 1, "few rows are one block");
    __shared__ __attribute__((aligned(1024))) char smem_raw[WAVES * (SLOT > MT * 1024 ? SLOT : MT * 1024)];
    LDS_AS char* slot = (LDS_AS char*)smem_raw + wave_id() * SLOT;
    const int lane = lane_id(), w = wave_id(), r = lane % 16, g = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int lr = lane / 8, lc = lane % 8;               // row and chunk that this lane loads
    const int kc = (g & 1) * 2 + (g >> 1);                // chunks kc and kc + 4 make its fragment
    const uint8_t* bsrc[2];
    const uint8_t* asrc[AL];
#pragma unroll
    for (int h = 0; h < 2; ++h) bsrc[h] = p.B + min(n0 + lr + 8 * h, (int64_t)p.N - 1) * p.ldb + 16 * lc;
#pragma unroll
    for (int h = 0; h < AL; ++h) asrc[h] = p.A + (int64_t)min(lr + 8 * h, p.M - 1) * p.lda + 16 * lc;   // rows past the end are not stored
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 b[DEPTH][2], a[DEPTH][AL];

    const int count = (p.K + kStep - 1) / kStep;           // steps; one past the last loads one line for all lanes
    auto first_byte = [&](int s) { return min((int64_t)s * kStep, (int64_t)p.K - kStep); };
    auto load = [&](int d, int s) {
        const int64_t k = first_byte(s);
#pragma unroll
        for (int h = 0; h < 2; ++h) b[d][h] = load16(s < count ? bsrc[h] + k : p.B);
#pragma unroll
        for (int h = 0; h < AL; ++h) a[d][h] = load16(s < count ? asrc[h] + k : p.A);
    };
    auto at = [&](int row, int c) { return reinterpret_cast<LDS_AS u32x4*>(slot + row * kStep + ((c ^ swz<8>(row)) << 4)); };
    auto multiply = [&](int d, int s) {
        const int had = (int)((int64_t)s * kStep - first_byte(s));   // bytes that earlier steps had
        if (had > 0) {
#pragma unroll
            for (int h = 0; h < AL; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int o = had - 16 * lc - 4 * q;
                    a[d][h][q] &= o >= 4 ? 0u : o <= 0 ? ~0u : ~0u << (8 * o);
                }
        }
        wave_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) *at(lr + 8 * h, lc) = b[d][h];
#pragma unroll
        for (int h = 0; h < AL; ++h) *at(16 + lr + 8 * h, lc) = a[d][h];
        wave_fence();
        const i32x8 fb = join16(*at(r, kc), *at(r, kc + 4));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = 16 + (FEW ? r % kFewRows : 16 * i + r);
            const i32x8 fa = join16(*at(row, kc), *at(row, kc + 4));
            acc[i] = mfma_f8<WIDE>(fb, fa, acc[i]);
        }
        __builtin_amdgcn_sched_barrier(0);   // steps mixed by the scheduler would not fit the registers
    };
    if (p.K >= kStep) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(d, w + d * WAVES);
        // (loads stand outside of branches: behind one, a wait for an older load would wait for them all)
        for (int s = w; s < count; s += DEPTH * WAVES)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (s + d * WAVES < count) multiply(d, s + d * WAVES);
                load(d, s + (d + DEPTH) * WAVES);
            }
    } else if (w == 0) {
        const uint8_t* brow = p.B + min(n0 + r, (int64_t)p.N - 1) * p.ldb;
        const i32x8 fb = join16(load_chunk(brow, 16 * g, p.K), load_chunk(brow, 64 + 16 * g, p.K));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint8_t* arow = p.A + (int64_t)min(16 * i + r, p.M - 1) * p.lda;
            acc[i] = mfma_f8<WIDE>(fb, join16(load_chunk(arow, 16 * g, p.K), load_chunk(arow, 64 + 16 * g, p.K)), acc[i]);
        }
    }
    lds_barrier();   // the slots are free
    auto part = [&](int q, int i, int l) { return reinterpret_cast<LDS_AS f32x4*>((LDS_AS char*)smem_raw + ((q * MT + i) * 64 + l) * 16); };
#pragma unroll
    for (int i = 0; i < MT; ++i) *part(w, i, lane) = acc[i];
    lds_barrier();
    for (int t = threadIdx.x; t < MT * 256; t += 64 * WAVES) {
        const int n = t % 16, m = t / 16;
        if (m >= p.M || n0 + n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) v += reinterpret_cast<LDS_AS float*>(part(q, m / 16, n / 4 * 16 + m % 16))[n % 4];
        store_c1(p.C, p.out_type, m * p.ldc + n0 + n, v * scale_or_one(p.sa, m) * scale_or_one(p.sb, n0 + n), p.alpha, p.beta);
    }
}

template <int MT, int WAVES, bool FEW>
hipError_t go(const F8Params& p, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.N + 15) / 16)), block(64 * WAVES);
    if (p.out_type == DT_F32) hipLaunchKernelGGL((f8_skinny_kernel<MT, WAVES, true, FEW>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((f8_skinny_kernel<MT, WAVES, false, FEW>), grid, block, 0, st, p);
    return hipGetLastError();
}

}  // namespace

// Expected microseconds: rounds of workgroups (the second one whole, later ones as waves come free), each a start and K's bytes;
// less on a half empty card (16 and 32 rows, N from 1000 to 128000, K from 512 to 14336; rows that are not 16-byte
// aligned on K = 2049 and 4097).
double f8_skinny_us(const F8Params& p) {
    const bool two = p.M > 16, aligned = ((uintptr_t)p.A | (uintptr_t)p.B | (uint64_t)p.lda | (uint64_t)p.ldb) % 16 == 0;
    const double all = (double)(((int64_t)p.N + 15) / 16) / num_compute_units(), rounds = all <= 0.5 ? 0.6 : all <= 1.0 ? 1.0 : all <= 2.0 ? 2.0 : all;
    const double round_us = two ? 2.0 + 0.85e-3 * p.K : 1.0 + 0.75e-3 * p.K;
    return 2.5 + rounds * round_us * (aligned ? 1.0 : two ? 1.7 : 1.5);
}

// Sixteen waves where eight would leave most of the card's wave slots empty and each still has steps to take.
hipError_t launch_f8_skinny(const F8Params& f, hipStream_t st) {
    if (f.M > kF8SkinnyRows) return hipErrorInvalidValue;
    return in_pieces(f, kF8SkinnyRows, kMostCols, [&](const F8Params& p) {
        const bool deep = ((int64_t)p.N + 15) / 16 <= 2 * num_compute_units() && p.K >= 2048;
        if (p.M <= kFewRows) return deep ? go<1, 16, true>(p, st) : go<1, 8, true>(p, st);
        if (p.M <= 16) return deep ? go<1, 16, false>(p, st) : go<1, 8, false>(p, st);
        return deep ? go<2, 16, false>(p, st) : go<2, 8, false>(p, st);
    });
}

}  // namespace gemm
