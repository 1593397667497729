// f8_common.hpp -- pieces of the 8-bit product's kernels: the matrix instruction, loads of
// K-contiguous rows of any pitch and length, and the scales.
#pragma once

#include "ops_common.hpp"

namespace gemm {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 x 16 += 16 x 128 times 128 x 16 in e4m3.  Each lane gives 32 bytes of row lane % 16 of either operand; the instruction
// sums over all of its k, so any assignment of k to lane groups and bytes serves as long as
// both operands use the same one.  Fed (B, A) it returns C transposed: lane l, register j
// holds C[m = l % 16][n = 4 * (l / 16) + j], four consecutive columns.
//
// Two forms.  The 8-bit instruction (v_mfma_f32_16x16x128_f8f6f4, unscaled) runs at twice
// the 16-bit rate, but does not sum in whole fp32: of each eight consecutive bytes of a lane it
// lines the products up with the largest and cuts them at 2^-13 of its power of two (measured
// by products of known size; the sums of eight are then added in fp32).  On random operands
// that is 1.5e-5 of the result: nothing beside a rounding to 16 bits (bf16 1.7e-3, f16
// 2.1e-4), but two hundred times an fp32 sum's error.  So fp32 results take the WIDE form, four
// v_mfma_f32_16x16x32_bf16 on the codes as bf16 (every e4m3 value is one), products exact
// and sums in fp32.
template <bool WIDE>
__device__ __forceinline__ f32x4 mfma_f8(i32x8 x, i32x8 y, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma_f8<false>(i32x8 x, i32x8 y, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, 0, 0, 0, 0);
}
// Eight e4m3 values (two words) as bf16.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
template <>
__device__ __forceinline__ f32x4 mfma_f8<true>(i32x8 x, i32x8 y, f32x4 c) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen((uint32_t)x[2 * q], (uint32_t)x[2 * q + 1]),
                                                    widen((uint32_t)y[2 * q], (uint32_t)y[2 * q + 1]), c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ i32x8 join16(u32x4 lo, u32x4 hi) {
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Bytes k .. k+15 of a row of K bytes, zeros past its end, reading nothing past it: the
// chunk that straddles the end is read as the row's last 16 bytes and shifted down.
__device__ __forceinline__ u32x4 load_chunk(const uint8_t* row, int k, int K) {
    if (k + 16 <= K) return load16(row + k);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k >= K) return v;
    if (K >= 16) {
        const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, load16(row + (K - 16)));
        return __builtin_bit_cast(u32x4, x >> (8 * (k + 16 - K)));
    }
    for (int i = k; i < K; ++i) v[(i - k) >> 2] |= (uint32_t)row[i] << (((i - k) & 3) * 8);
    return v;
}

// A result is (sum * scale_a) * scale_b: the product of the scales alone may leave fp32's range where the result does not.
__device__ __forceinline__ float scale_or_one(const float* s, int64_t i) { return s ? s[i] : 1.0f; }

}  // namespace gemm
