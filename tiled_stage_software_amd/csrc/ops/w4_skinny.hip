// w4_skinny.hip -- C = alpha * A * W^T + beta * C with W[n][k] = s * (q - z): 4-bit codes q,
// two to a byte, and a scale s and zero point z for each row n and group of k.
//
// By groups:  sum_k a * s * (q - z) = s * (sum_k a * q - z * sum_k a), the sums on the matrix
// cores in fp32.  A code becomes a 16-bit float with two operations a pair: q placed at the
// top of the mantissa of 1.0 is exactly 1 + q/16, so
//   sum a*(q - z) = 16 * (sum a*(1 + q/16) - (1 + z/16) * sum a),
// and the sum of a, one instruction against ones, serves every column.  No weight is rounded:
// the scale multiplies the fp32 sum of its group.
//
// Few rows of A: the codes' bytes bound it.  A workgroup computes 16 columns, its eight waves
// share K; every lane loads its own 16 bytes (32 codes) of a row straight into registers as
// the matrix instruction's second operand, with no LDS between.
#include "ops_common.hpp"

namespace gemm {
namespace {

template <int T> struct Half;
template <> struct Half<DT_BF16> {
    static constexpr uint32_t ONES = 0x3F803F80u;   // 1.0, twice
    static constexpr int TOP = 3;                   // the code's place at the top of the mantissa
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <> struct Half<DT_F16> {
    static constexpr uint32_t ONES = 0x3C003C00u;
    static constexpr int TOP = 6;
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

// Eight codes as 1 + q/16: result i holds codes i and i + 4 in its halves.
template <int T>
__device__ __forceinline__ u32x4 spread(uint32_t w) {
    constexpr int TOP = Half<T>::TOP;
    constexpr uint32_t MASK = 0x000F000Fu << TOP;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = 4 * i - TOP;
        v[i] = ((s < 0 ? w << -s : w >> s) & MASK) | Half<T>::ONES;
    }
    return v;
}
// Eight elements of A in the order spread() gives the codes: 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ u32x4 shuffle8(u32x4 a) {
    u32x4 v;
    v[0] = __builtin_amdgcn_perm(a[2], a[0], 0x05040100u);
    v[1] = __builtin_amdgcn_perm(a[2], a[0], 0x07060302u);
    v[2] = __builtin_amdgcn_perm(a[3], a[1], 0x05040100u);
    v[3] = __builtin_amdgcn_perm(a[3], a[1], 0x07060302u);
    return v;
}

// Eight elements of a row of K from k, zeros past its end.
__device__ __forceinline__ u32x4 load_a(const char* row, int k, int K) {
    if (k + 8 <= K) return load16(row + (int64_t)k * 2);
    u32x4 v = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 8; ++i)
        if (k + i < K) v[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[k + i] << ((i & 1) * 16);
    return v;
}
// Eight codes (four bytes) from k; what lies past the row's bytes is not read.  (Codes past
// K meet zeros of A.)
__device__ __forceinline__ uint32_t load_q(const uint8_t* row, int k, int K) {
    uint32_t v = 0;
    if (k + 8 <= K) {
        __builtin_memcpy(&v, row + (k >> 1), 4);
        return v;
    }
    for (int i = 0; i < 4; ++i)
        if (k + 2 * i < K) v |= (uint32_t)row[(k >> 1) + i] << (8 * i);
    return v;
}

// 16 columns and MT x 16 rows per workgroup; a step is 32 k, which one group holds.
constexpr int kWaves = 8;
template <int T, int MT>
__global__ __launch_bounds__(64 * kWaves) void w4_simple_kernel(const W4Params p, int tiles_n) {
    __shared__ float part[kWaves][MT][64][4];
    const int lane = lane_id(), w = wave_id(), r = lane % 16, g = lane / 16;
    const int n0 = (int)(blockIdx.x % tiles_n) * 16, m0 = (int)(blockIdx.x / tiles_n) * 16 * MT;
    const int nc = min(n0 + r, p.N - 1);
    const uint8_t* qrow = p.W + (int64_t)nc * p.ldw;
    const char* arow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) arow[i] = p.A + (int64_t)min(m0 + 16 * i + r, p.M - 1) * p.lda * 2;
    const u32x4 ones = {Half<T>::ONES, Half<T>::ONES, Half<T>::ONES, Half<T>::ONES};
    f32x4 total[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) total[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = (p.K + 31) / 32;
    for (int s = w; s < steps; s += kWaves) {
        const int k = s * 32 + 8 * g;
        const u32x4 b = spread<T>(load_q(qrow, k, p.K));
        const int64_t gi = (int64_t)nc * p.lds + s * 32 / p.group;
        const float sc = 16.0f * load_elem(p.scales, T, gi);
        const float z1 = -1.0f - (p.zeros ? load_elem(p.zeros, T, gi) : 8.0f) * 0.0625f;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const u32x4 a = shuffle8(load_a(arow[i], k, p.K));
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            const f32x4 dot = Half<T>::mfma(a, b, zero), sum = Half<T>::mfma(a, ones, zero);
#pragma unroll
            for (int e = 0; e < 4; ++e) total[i][e] = __builtin_fmaf(sc, __builtin_fmaf(z1, sum[e], dot[e]), total[i][e]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[w][i][lane][e] = total[i][e];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 256; t += 64 * kWaves) {
        const int i = t / 256, l = t % 64, e = t / 64 % 4;
        const int m = m0 + 16 * i + 4 * (l / 16) + e, col = n0 + l % 16;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) v += part[q][i][l][e];
        if (m < p.M && col < p.N) store_c1(p.C, p.out_type, (int64_t)m * p.ldc + col, v, p.alpha, p.beta);
    }
}

template <int T, int MT>
hipError_t go(const W4Params& p, hipStream_t st) {
    const int64_t tn = ((int64_t)p.N + 15) / 16, tm = ((int64_t)p.M + 16 * MT - 1) / (16 * MT);
    if (tm * tn > INT32_MAX / (64 * kWaves)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((w4_simple_kernel<T, MT>), dim3((unsigned)(tm * tn)), dim3(64 * kWaves), 0, st, p, (int)tn);
    return hipGetLastError();
}

template <int T>
hipError_t skinny_of(const W4Params& p, hipStream_t st) {
    return p.M <= 16 ? go<T, 1>(p, st) : go<T, 4>(p, st);
}

}  // namespace

hipError_t launch_w4_skinny(int in_type, const W4Params& p, hipStream_t st) {
    return in_type == DT_BF16 ? skinny_of<DT_BF16>(p, st) : skinny_of<DT_F16>(p, st);
}

}  // namespace gemm
