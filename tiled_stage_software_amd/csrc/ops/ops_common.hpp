// ops_common.hpp -- device helpers shared by the operators' kernels.
#pragma once

#include "ops.hpp"

namespace gemm {

// 16 bytes at any address: the target serves unaligned global vectors, so rows of any pitch
// use the same instruction as aligned ones.
__device__ __forceinline__ u32x4 load16(const void* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// Orders a wave's own LDS writes and reads for the compiler (the hardware keeps their order).
__device__ __forceinline__ void wave_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}
// Barrier for what the workgroup shares in LDS; unlike __syncthreads() it leaves loads from memory in flight.
__device__ __forceinline__ void lds_barrier() {
    wait_lgkm0();
    barrier();
}

template <int T>
__device__ __forceinline__ float to_f32(uint16_t b) {
    return T == DT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}
template <int T>
__device__ __forceinline__ uint16_t from_f32(float v) {
    return T == DT_BF16 ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
}

template <int T>
struct Elem {  // elements of a 16-byte vector
    static constexpr int SIZE = T == DT_F32 ? 4 : 2;
    static constexpr int VE = 16 / SIZE;
    static __device__ __forceinline__ float get(const u32x4& v, int e) {
        if constexpr (T == DT_F32) return __uint_as_float(v[e]);
        else return to_f32<T>((uint16_t)(v[e >> 1] >> ((e & 1) * 16)));
    }
    static __device__ __forceinline__ u32x4 pack(const float* f) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == DT_F32) v[i] = __float_as_uint(f[i]);
            else v[i] = (uint32_t)from_f32<T>(f[2 * i]) | ((uint32_t)from_f32<T>(f[2 * i + 1]) << 16);
        }
        return v;
    }
};

// Element i of an array of 16- or 32-bit floats whose type is known at run time.
__device__ __forceinline__ float load_elem(const char* p, int type, int64_t i) {
    if (type == DT_F32) return reinterpret_cast<const float*>(p)[i];
    const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
    return type == DT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// Four floats to four e4m3 codes, round to nearest even (v_cvt_pk_fp8_f32: OCP codes on
// this target; NaN stays NaN).  The callers' values are at most 448 but for a rounding.
__device__ __forceinline__ uint32_t pack_f8x4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// Sum / largest bits over the 64 lanes of a wave, in every lane, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, s, 64);
        v = o > v ? o : v;
    }
    return v;
}

// 1 / sqrt(sum / cols + eps) from the row's sum of squares.  Where that sum leaves fp32's range
// though the row does not (|h| above 2^64 / sqrt(cols); |h| below 2^-45 with so small an eps), `again` sums
// the squares of h * 2^-80 or h * 2^80, which stay in range for any such row.
template <class F>
__device__ __forceinline__ float row_rstd(float sum, int cols, float eps, F&& again) {
    const float mean = sum / (float)cols + eps;
    const bool high = __builtin_isinf(sum);
    if (high || mean < 0x1p-90f) {   // the same in every thread of the row
        const float by = high ? 0x1p-80f : 0x1p80f;
        return by / __builtin_sqrtf(again(by) / (float)cols + eps * by * by);
    }
    return 1.0f / __builtin_sqrtf(mean);
}

// Launches of a product's kernel for at most `rows` x `cols` of C each: grids are counted in 32 bits, workgroups times
// threads, and have 65535 rows at most, which sizes up to 2^30 can pass.
constexpr int64_t kMostCols = int64_t(1) << 24;
inline void skip(F8Params& p, int64_t m, int64_t n) {
    p.A += m * p.lda;
    p.B += n * p.ldb;
    if (p.sa) p.sa += m;
    if (p.sb) p.sb += n;
}
inline void skip(W4Params& p, int64_t m, int64_t n) {
    p.A += m * p.lda * 2;
    p.W += n * p.ldw;
    p.scales += n * p.lds * 2;
    if (p.zeros) p.zeros += n * p.lds * 2;
}
template <class P, class Launch>
hipError_t in_pieces(const P& p, int64_t rows, int64_t cols, Launch&& launch) {
    for (int64_t m = 0; m < p.M; m += rows)
        for (int64_t n = 0; n < p.N; n += cols) {
            P q = p;
            skip(q, m, n);
            q.C += (m * p.ldc + n) * (p.out_type == DT_F32 ? 4 : 2);
            q.M = (int)(p.M - m < rows ? p.M - m : rows);
            q.N = (int)(p.N - n < cols ? p.N - n : cols);
            const hipError_t e = launch(q);
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

// One element of C = alpha * acc + beta * C (beta == 0: C is not read).
__device__ __forceinline__ void store_c1(char* C, int out_type, int64_t at, float acc, float alpha, float beta) {
    if (out_type == DT_F32) {
        float* c = reinterpret_cast<float*>(C) + at;
        *c = epi(acc, alpha, beta, beta != 0.0f ? *c : 0.0f);
    } else {
        uint16_t* c = reinterpret_cast<uint16_t*>(C) + at;
        const bool bf = out_type == DT_BF16;
        const float o = beta != 0.0f ? (bf ? bf16_bits_to_f32(*c) : f16_bits_to_f32(*c)) : 0.0f;
        const float v = epi(acc, alpha, beta, o);
        *c = bf ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
    }
}

}  // namespace gemm
