// w4_common.hpp -- the arithmetic of 4-bit weights.
//
// W[n][k] = s * (q - z) with a scale s and zero point z for each row n and group of k.  By groups:
//   sum_k a * s * (q - z) = s * (sum_k a * q - z * sum_k a),
// the sums on the matrix cores in fp32.  A code becomes a 16-bit float by placing it at the
// top of the mantissa of 1.0, which is exactly 1 + q/16, so
//   sum a*(q - z) = 16 * (sum a*(1 + q/16) - (1 + z/16) * sum a).
// No weight is rounded: the scale multiplies the fp32 sum of its group.
#pragma once

#include "ops_common.hpp"

namespace gemm {

template <int T> struct Half;
template <> struct Half<DT_BF16> {
    typedef __bf16 type;
    static constexpr uint32_t ONES = 0x3F803F80u;   // 1.0, twice
    static constexpr int TOP = 3;                   // the code's place at the top of the mantissa
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <> struct Half<DT_F16> {
    typedef _Float16 type;
    static constexpr uint32_t ONES = 0x3C003C00u;
    static constexpr int TOP = 6;
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

// Turns codes into operands.  The mask and the ones sit in registers, out of the compiler's sight, so that
// masking and joining are one v_and_or_b32 (as literals they are two instructions).
template <int T>
struct Spread {
    static constexpr int TOP = Half<T>::TOP;
    uint32_t mask, ones, twice;
    __device__ __forceinline__ Spread() : mask(0x000F000Fu << TOP), ones(Half<T>::ONES), twice(0x1001u << TOP) {
        asm("" : "+s"(mask));
        asm("" : "+v"(ones));
        asm("" : "+v"(twice));
    }
    __device__ __forceinline__ uint32_t place(uint32_t v) const { return (v & mask) | ones; }
    // Eight codes (code i in bits 4 i .. 4 i + 3) in their order: byte i times 2^TOP + 2^(12 + TOP) has code 2 i at bit TOP and
    // code 2 i + 1 at bit 16 + TOP, and the mask drops the rest.  Eight operations, the byte chosen by the product's operand.
    __device__ __forceinline__ u32x4 in_order(uint32_t w) const {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = place(__umul24((w >> 8 * i) & 0xFF, twice));
        return v;
    }
    // The same as pairs (0, 4), (1, 5), (2, 6), (3, 7), for an A whose eight elements lie so: eight operations.
    __device__ __forceinline__ u32x4 in_pairs(uint32_t w) const {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = place(4 * i < TOP ? w << (TOP - 4 * i) : w >> (4 * i - TOP));
        return v;
    }
};
// Eight 16-bit elements in the order of in_pairs().
__device__ __forceinline__ u32x4 pairs_of(u32x4 a) {
    return u32x4{__builtin_amdgcn_perm(a[2], a[0], 0x05040100u), __builtin_amdgcn_perm(a[2], a[0], 0x07060302u),
                 __builtin_amdgcn_perm(a[3], a[1], 0x05040100u), __builtin_amdgcn_perm(a[3], a[1], 0x07060302u)};
}

// 1 + z/16 of a group.
template <int T>
__device__ __forceinline__ float zero16(uint16_t z) { return 1.0f + to_f32<T>(z) * 0.0625f; }
constexpr float kZero16 = 1.5f;   // of z = 8

// Bytes of a chunk moved down by `by`, zeros behind them (16 or more: all zeros).
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int by) {
    if (by >= 16) return u32x4{0u, 0u, 0u, 0u};
    return __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, v) >> (8 * by));
}
// Eight elements of a row of K from k, zeros past its end.  Those across or past it are read as the row's last eight and moved
// down: one load whatever k is, none behind a branch.
__device__ __forceinline__ u32x4 load_a(const char* row, int k, int K) {
    if (K >= 8) {
        const int at = min(k, K - 8);
        const u32x4 v = load16(row + (int64_t)at * 2);
        return k == at ? v : shift_down(v, 2 * (k - at));
    }
    u32x4 v = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 8; ++i)
        if (k + i < K) v[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[k + i] << ((i & 1) * 16);
    return v;
}
// Eight codes (four bytes) from k, zeros past the row's bytes, in the same way.  (Codes past K meet zeros of A.)
__device__ __forceinline__ uint32_t load_q(const uint8_t* row, int k, int K) {
    const int bytes = (K + 1) >> 1;
    uint32_t v = 0;
    if (bytes >= 4) {
        const int at = min(k >> 1, bytes - 4), by = (k >> 1) - at;
        __builtin_memcpy(&v, row + at, 4);
        return by >= 4 ? 0u : v >> (8 * by);
    }
    for (int i = 0; i < 4; ++i)
        if (k + 2 * i < K) v |= (uint32_t)row[(k >> 1) + i] << (8 * i);
    return v;
}

// The same for 32 codes (16 bytes).
__device__ __forceinline__ u32x4 load_q16(const uint8_t* row, int k, int K) {
    const int bytes = (K + 1) >> 1;
    if (bytes >= 16) {
        const int at = min(k >> 1, bytes - 16);
        return shift_down(load16(row + at), (k >> 1) - at);
    }
    return u32x4{load_q(row, k, K), load_q(row, k + 8, K), load_q(row, k + 16, K), load_q(row, k + 24, K)};
}

}  // namespace gemm
