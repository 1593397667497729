// linear_skinny.hip -- the product with bias, activation and residual for few rows of A: W's bytes bound it.
//
// As the 8-bit product's kernel for few rows: a workgroup computes 16 columns (MT x 16 rows); its waves share K, each taking
// every WAVES-th step of 64 elements (128 bytes of a row), DEPTH steps of loads ahead of the one it multiplies.  Eight lanes load
// 128 consecutive bytes of a row, which the address unit takes at its full rate, and a slot of LDS that belongs to the wave
// turns them into the matrix instruction's fragments: no barrier, the wave's LDS operations run in order.  A goes the
// same way; FEW: at most kFewRows rows, a quarter of the loads.
//
// 1 x 14336 x 4096 bf16 with gelu: 23.3 us, 5.0 TB/s.
//
// A last step that K does not fill is the row's last 128 bytes, with zeros in A and in W for what earlier steps had (an infinity
// there times a zero would be NaN).  The waves' sums meet in LDS in wave order.
#include "f8_common.hpp"
#include "linear.hpp"

namespace gemm {
namespace {

constexpr int kStep = 128, kFewRows = 4;   // bytes

template <int T>
__device__ __forceinline__ f32x4 mfma16(u32x4 w, u32x4 a, f32x4 c) {
    typedef typename Mfma<half_of<T>, 16>::frag frag;
    return Mfma<half_of<T>, 16>::run(__builtin_bit_cast(frag, w), __builtin_bit_cast(frag, a), c);
}

template <int T, int OUT, int MT, int WAVES, bool FEW>
__global__ __launch_bounds__(64 * WAVES) void linear_skinny_kernel(const LinearParams p, const LinearEpi e) {
    constexpr int DEPTH = MT == 1 || WAVES == 8 ? 4 : 2;   // what the registers hold
    constexpr int AL = FEW ? 1 : 2 * MT;                  // 16-byte loads of A per step, eight rows each
    constexpr int SLOT = (16 + 8 * AL) * kStep;
    static_assert(!FEW || MT == 1, "few rows are one block");
    __shared__ __attribute__((aligned(1024))) char smem_raw[WAVES * (SLOT > MT * 1024 ? SLOT : MT * 1024)];
    LDS_AS char* slot = (LDS_AS char*)smem_raw + wave_id() * SLOT;
    const int lane = lane_id(), w = wave_id(), r = lane % 16, g = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int lr = lane / 8, lc = lane % 8;               // row and chunk that this lane loads
    const int kc = (g & 1) * 2 + (g >> 1);                // chunks kc and kc + 4 are its two fragments
    const int64_t K = 2 * (int64_t)p.K;                   // bytes of a row
    const char* wsrc[2];
    const char* asrc[AL];
#pragma unroll
    for (int h = 0; h < 2; ++h) wsrc[h] = p.W + min(n0 + lr + 8 * h, (int64_t)p.N - 1) * p.ldw * 2 + 16 * lc;
#pragma unroll
    for (int h = 0; h < AL; ++h) asrc[h] = p.A + (int64_t)min(lr + 8 * h, p.M - 1) * p.lda * 2 + 16 * lc;   // rows past the end are not stored
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 b[DEPTH][2], a[DEPTH][AL];

    const int64_t count = (K + kStep - 1) / kStep;         // steps; one past the last loads one line for all lanes
    auto first_byte = [&](int64_t s) { return min(s * kStep, K - kStep); };
    auto load = [&](int d, int64_t s) {
        const int64_t k = first_byte(s);
#pragma unroll
        for (int h = 0; h < 2; ++h) b[d][h] = load16(s < count ? wsrc[h] + k : p.W);
#pragma unroll
        for (int h = 0; h < AL; ++h) a[d][h] = load16(s < count ? asrc[h] + k : p.A);
    };
    auto at = [&](int row, int c) { return reinterpret_cast<LDS_AS u32x4*>(slot + row * kStep + ((c ^ swz<8>(row)) << 4)); };
    auto multiply = [&](int d, int64_t s) {
        const int had = (int)(s * kStep - first_byte(s));   // bytes that earlier steps had
        if (had > 0) {
            u32x4 mask;   // the same chunk of every row
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int o = had - 16 * lc - 4 * q;
                mask[q] = o >= 4 ? 0u : o <= 0 ? ~0u : ~0u << (8 * o);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) b[d][h] &= mask;
#pragma unroll
            for (int h = 0; h < AL; ++h) a[d][h] &= mask;
        }
        wave_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) *at(lr + 8 * h, lc) = b[d][h];
#pragma unroll
        for (int h = 0; h < AL; ++h) *at(16 + lr + 8 * h, lc) = a[d][h];
        wave_fence();
        const u32x4 f0 = *at(r, kc), f1 = *at(r, kc + 4);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = 16 + (FEW ? r % kFewRows : 16 * i + r);
            acc[i] = mfma16<T>(f0, *at(row, kc), acc[i]);
            acc[i] = mfma16<T>(f1, *at(row, kc + 4), acc[i]);
        }
        __builtin_amdgcn_sched_barrier(0);   // steps mixed by the scheduler would not fit the registers
    };
    if (K >= kStep) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(d, w + d * WAVES);
        // (loads stand outside of branches: behind one, a wait for an older load would wait for them all)
        for (int64_t s = w; s < count; s += DEPTH * WAVES)
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (s + d * WAVES < count) multiply(d, s + d * WAVES);
                load(d, s + (d + DEPTH) * WAVES);
            }
    } else if (w == 0) {
        auto chunk = [&](const char* base, int64_t row, int64_t ld, int k) {
            return load_chunk(reinterpret_cast<const uint8_t*>(base) + row * ld * 2, k, (int)K);
        };
        const int64_t wr = min(n0 + r, (int64_t)p.N - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 f = chunk(p.W, wr, p.ldw, 64 * h + 16 * g);
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] = mfma16<T>(f, chunk(p.A, min(16 * i + r, p.M - 1), p.lda, 64 * h + 16 * g), acc[i]);
        }
    }
    lds_barrier();   // the slots are free
    auto part = [&](int q, int i, int l) { return reinterpret_cast<LDS_AS f32x4*>((LDS_AS char*)smem_raw + ((q * MT + i) * 64 + l) * 16); };
#pragma unroll
    for (int i = 0; i < MT; ++i) *part(w, i, lane) = acc[i];
    // eight columns of a row a thread: what it adds to them is on its way before the sums are there
    const int t = threadIdx.x, m = t / 2, n = (int)n0 + 8 * (t % 2);
    const bool mine = t < MT * 32 && m < p.M && n < p.N;
    float bias[8];
    Eight<OUT> old;
    if (mine) {
        load_bias<T>(e, n, bias);
        if (e.R) old.load(e.R + m * e.ldr * Elem<OUT>::SIZE, n, p.N);
    }
    lds_barrier();
    if (!mine) return;
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < WAVES; ++q) s += *part(q, m / 16, (2 * (t % 2) + h) * 16 + m % 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[4 * h + q] = s[q];
    }
    finish8<T, OUT>(e, m, n, 0, v, bias, old);
}

template <int MT, int WAVES, bool FEW>
hipError_t go(int in_type, const LinearParams& p, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.N + 15) / 16)), block(64 * WAVES);
    return by_type(in_type, p.out_type, [&](auto t, auto o) {
        hipLaunchKernelGGL((linear_skinny_kernel<decltype(t)::value, decltype(o)::value, MT, WAVES, FEW>), grid, block, 0, st, p, epi_of(p));
        return hipGetLastError();
    });
}

}  // namespace

// Sixteen waves where eight would leave most of the card's wave slots empty and each still has steps to take.
hipError_t launch_linear_skinny(int in_type, const LinearParams& f, hipStream_t st) {
    if (f.M > kLinearSkinnyRows || f.K < 1) return hipErrorInvalidValue;
    return in_pieces(f, kLinearSkinnyRows, kMostCols, [&](const LinearParams& p) {
        const bool deep = ((int64_t)p.N + 15) / 16 <= 2 * num_compute_units() && p.K >= 1024;
        if (p.M <= kFewRows) return deep ? go<1, 16, true>(in_type, p, st) : go<1, 8, true>(in_type, p, st);
        if (p.M <= 16) return deep ? go<1, 16, false>(in_type, p, st) : go<1, 8, false>(in_type, p, st);
        return deep ? go<2, 16, false>(in_type, p, st) : go<2, 8, false>(in_type, p, st);
    });
}

}  // namespace gemm
