// linear.hpp -- what the kernels of the product with bias, activation and residual share: the
// activations with their derivatives, and the epilogue.
//
//   C = act(A W^T + bias) + R,  Z = A W^T + bias
//
// The epilogue works in fp32 on eight consecutive columns of a row at a time, which a thread takes from the workgroup's
// sums in LDS (or from the splits' sums in memory): bias, R, Z and C then move in whole vectors, neighbouring
// threads along a row, and a thread keeps its columns, so it loads their bias once.  In the accumulators' own layout a lane
// has four columns of one row, and R would be read in pieces of 8 bytes from 16 rows an instruction.  Z is rounded
// once from the sum with its bias; C is computed from the same unrounded value and rounded once.
#pragma once

#include "../mfma.hpp"
#include "ops_common.hpp"

namespace gemm {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

template <int T>
using half_of = std::conditional_t<T == DT_BF16, __bf16, _Float16>;

struct LinearEpi {
    const char* bias;    // N, or NULL
    const char* R;       // C's type, or NULL
    char* Z;             // the operands' type, or NULL
    char* C;
    int64_t ldr, ldz, ldc;
    int M, N;
    int bias_type, act;
};

// ------------------------------------------------------------------ activations
// 1 / (1 + exp(-q)) from q * log2(e).  exp2 passes to infinity and its reciprocal to 0 where the result does.
__device__ __forceinline__ float sigmoid_of(float q_log2e) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-q_log2e)); }

constexpr float kLog2e = 1.4426950408889634f;
// gelu(z), tanh form: z / (1 + exp(-2 sqrt(2/pi) (z + 0.044715 z^3)))
constexpr float kTanh1 = 2.302208198f, kTanh3 = 0.1029432397f;   // 2 sqrt(2/pi) log2(e), and 0.044715 times that

// The upper tail of the normal distribution at a >= 0, 1 - Phi(a) = exp(-a^2 / 2) * t * P(t), t = 1 / (1 + 0.23 a): P is the
// polynomial of degree 7 with the least largest relative error for a up to 13 (1.3e-7; 5e-7 with fp32 steps),
// fitted here by reweighted least squares.  bell: exp(-a^2 / 2).
__device__ __forceinline__ float upper_tail(float a, float& bell) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.23f, a, 1.0f));
    bell = __builtin_amdgcn_exp2f(a * a * (-0.5f * kLog2e));
    float p = -0.07388245619f;
    p = __builtin_fmaf(p, t, 0.2688493705f);
    p = __builtin_fmaf(p, t, -0.2349846766f);
    p = __builtin_fmaf(p, t, 0.2535974279f);
    p = __builtin_fmaf(p, t, -0.0007328644353f);
    p = __builtin_fmaf(p, t, 0.1061034937f);
    p = __builtin_fmaf(p, t, 0.08914202063f);
    p = __builtin_fmaf(p, t, 0.09190775127f);
    return bell * t * p;
}

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;   // (NaN stays)
    // (the least z: its sigmoid, or tail, is 0, which an infinity would meet; where z is NaN the other factor stays one)
    if constexpr (ACT == ACT_GELU) {
        float bell;
        const float a = __builtin_fminf(__builtin_fabsf(z), 40.0f);
        const float low = a * upper_tail(a, bell);   // |z| (1 - Phi(|z|))
        return z < 0.0f ? -low : z - low;
    }
    if constexpr (ACT == ACT_GELU_TANH) return __builtin_fmaxf(z, -1e4f) * sigmoid_of(z * __builtin_fmaf(kTanh3, z * z, kTanh1));
    if constexpr (ACT == ACT_SILU) return __builtin_fmaxf(z, -1e4f) * sigmoid_of(z * kLog2e);
    return z;
}
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : z == z ? 0.0f : z;
    if constexpr (ACT == ACT_NONE) return 1.0f;
    // past these the slope is 0 or 1 in fp32, and products of z would meet infinities
    z = z > 60.0f ? 60.0f : z < -120.0f ? -120.0f : z;   // (NaN stays)
    if constexpr (ACT == ACT_GELU) {
        float bell;
        const float tail = upper_tail(__builtin_fabsf(z), bell);
        return __builtin_fmaf(z * 0.3989422804f, bell, z < 0.0f ? tail : 1.0f - tail);   // Phi(z) + z phi(z)
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float s = sigmoid_of(z * __builtin_fmaf(kTanh3, z * z, kTanh1));
        const float d = z * __builtin_fmaf(3.0f * 0.07135481283f, z * z, 1.595769122f);   // z times the inner derivative
        return __builtin_fmaf(d, s * (1.0f - s), s);
    }
    const float s = sigmoid_of(z * kLog2e);
    return __builtin_fmaf(z, s * (1.0f - s), s);
}
template <int N>
__device__ __forceinline__ void act_all(int act, float (&v)[N]) {
    switch (act) {   // the same for the whole launch
        case ACT_RELU:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_of<ACT_RELU>(v[e]);
            break;
        case ACT_GELU:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_of<ACT_GELU>(v[e]);
            break;
        case ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_of<ACT_GELU_TANH>(v[e]);
            break;
        case ACT_SILU:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_of<ACT_SILU>(v[e]);
            break;
    }
}

// ------------------------------------------------------------------ eight columns of a row
// Columns n .. n+7 of a row that starts at `row`; those from N on are 0 and not read (n < N).  Where they are not whole they come one
// by one, none behind a branch: waits between them would be a load's latency each.
template <int T>
struct Eight {
    static constexpr int Q = T == DT_F32 ? 2 : 1;
    u32x4 raw[Q];
    __device__ __forceinline__ void whole(const char* row, int n) {
#pragma unroll
        for (int q = 0; q < Q; ++q) raw[q] = load16(row + (int64_t)n * Elem<T>::SIZE + 16 * q);
    }
    __device__ __forceinline__ void load(const char* row, int n, int N) {
        if (n + 8 <= N) {
            whole(row, n);
            return;
        }
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = min(n + e, N - 1);
            if constexpr (T == DT_F32) x[e] = reinterpret_cast<const uint32_t*>(row)[at];
            else x[e] = reinterpret_cast<const uint16_t*>(row)[at];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = n + e < N ? x[e] : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (T == DT_F32) raw[0][e] = x[e], raw[1][e] = x[4 + e];
            else raw[0][e] = x[2 * e] | x[2 * e + 1] << 16;
        }
    }
    __device__ __forceinline__ float get(int e) const { return Elem<T>::get(raw[e / Elem<T>::VE], e % Elem<T>::VE); }
};
// Eight values to columns n .. n+7, those within [lo, N).
template <int T>
__device__ __forceinline__ void store8(char* row, int n, int lo, int N, const float* v) {
    constexpr int SZ = Elem<T>::SIZE, VE = Elem<T>::VE;
    if (n >= lo && n + 8 <= N) {
#pragma unroll
        for (int q = 0; q < 8 / VE; ++q) store16(row + (int64_t)n * SZ + 16 * q, Elem<T>::pack(v + VE * q));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (n + e >= lo && n + e < N) {
            if constexpr (T == DT_F32) reinterpret_cast<float*>(row)[n + e] = v[e];
            else reinterpret_cast<uint16_t*>(row)[n + e] = from_f32<T>(v[e]);
        }
}

// Bias of columns n .. n+7 (0 where there is none).
template <int T>
__device__ __forceinline__ void load_bias(const LinearEpi& e, int n, float* b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.0f;
    if (!e.bias || n >= e.N) return;
    if (e.bias_type == DT_F32) {
        Eight<DT_F32> v;
        v.load(e.bias, n, e.N);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = v.get(i);
    } else {
        Eight<T> v;
        v.load(e.bias, n, e.N);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = v.get(i);
    }
}
// From the sums v of columns n .. n+7 in row m to Z and C (those within [lo, N)); `old`: R's.
template <int T, int OUT>
__device__ __forceinline__ void finish8(const LinearEpi& e, int64_t m, int n, int lo, float (&v)[8], const float* bias,
                                        const Eight<OUT>& old) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += bias[i];
    if (e.Z) store8<T>(e.Z + m * e.ldz * 2, n, lo, e.N, v);
    act_all(e.act, v);
    if (e.R) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += old.get(i);
    }
    store8<OUT>(e.C + m * e.ldc * Elem<OUT>::SIZE, n, lo, e.N, v);
}

// Sums of a BM x BN tile from the accumulators of NT threads through LDS (`bytes` of it, free once every wave has arrived) to
// Z and C.  The tile's rows from m_keep and columns from n_keep on, within M and N, are stored.  As many of each wave's block
// rows as LDS holds go through at a time; a row's 16-byte chunk c lies at c ^ (row mod 16), so that the 16 rows
// which a write touches, and the chunks of a row which a read does, spread over the banks.
template <int T, int OUT, int BM, int BN, int WM, int WN, int MI, int BYTES, class Compute>
__device__ __forceinline__ void linear_epilogue(Compute& ops, const LinearEpi& e, LDS_AS char* smem, int m0, int n0, int m_keep,
                                                int n_keep) {
    constexpr int NT = 64 * WM * WN, WTM = BM / WM, WTN = BN / WN, TM = WTM / MI, TN = WTN / MI, NR = MI * MI / 64;
    constexpr int ROWB = BN * 4, FIT = BYTES / (ROWB * MI * WM);
    constexpr int BLK = FIT >= TM ? TM : FIT;           // block rows of a wave in one pass
    static_assert(BLK >= 1 && BN >= 64 && (BN & (BN - 1)) == 0 && NT % (BN / 8) == 0, "whole rows of chunks");
    constexpr int TPR = BN / 8, RPI = NT / TPR;         // threads of a row, rows at a time
    const int w = wave_id(), wm = w / WN, wn = w % WN, lane = lane_id();
    const int c8 = (int)threadIdx.x % TPR, n = n0 + 8 * c8;
    float bias[8];
    load_bias<T>(e, n, bias);
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += BLK) {
        constexpr int ROWS = WM * BLK * MI;
        wait_lgkm0();
        barrier();   // LDS is free
#pragma unroll
        for (int i = 0; i < BLK; ++i) {
            if (i0 + i >= TM) continue;
            const int r = (wm * BLK + i) * MI + lane % MI;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < NR / 4; ++g) {
                    const int c = (wn * WTN + j * MI + g * 8 + (lane / MI) * 4) / 4;
                    f32x4 v;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = ops.acc[i0 + i][j][4 * g + q];
                    *reinterpret_cast<LDS_AS f32x4*>(smem + r * ROWB + ((c ^ (r & 15)) << 4)) = v;
                }
        }
        wait_lgkm0();
        barrier();
        auto row_of = [&](int s) { return m0 + s / (BLK * MI) * WTM + i0 * MI + s % (BLK * MI); };
        auto mine = [&](int s) {
            const int m = row_of(s);
            return s < ROWS && (TM % BLK == 0 || i0 + s % (BLK * MI) / MI < TM) && m >= m_keep && m < e.M && n < e.N && n + 8 > n_keep;
        };
        // R of four rows is on its way before the first of them is stored, which the compiler could not move it past
        constexpr int AHEAD = 4;
        for (int s0 = (int)threadIdx.x / TPR; s0 < ROWS; s0 += AHEAD * RPI) {
            Eight<OUT> old[AHEAD];
            if (e.R) {
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    const int s = s0 + a * RPI;
                    if (mine(s)) old[a].load(e.R + (int64_t)row_of(s) * e.ldr * Elem<OUT>::SIZE, n, e.N);
                }
            }
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int s = s0 + a * RPI;
                if (!mine(s)) continue;
                float v[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 x = *reinterpret_cast<LDS_AS const f32x4*>(smem + s * ROWB + (((2 * c8 + h) ^ (s & 15)) << 4));
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[4 * h + q] = x[q];
                }
                finish8<T, OUT>(e, row_of(s), n, n_keep, v, bias, old[a]);
            }
        }
    }
}

// ------------------------------------------------------------------ launches
inline void skip(LinearParams& p, int64_t m, int64_t n) {
    p.A += m * p.lda * 2;
    p.W += n * p.ldw * 2;
    if (p.bias) p.bias += n * (p.bias_type == DT_F32 ? 4 : 2);
    if (p.R) p.R += (m * p.ldr + n) * (p.out_type == DT_F32 ? 4 : 2);
    if (p.Z) p.Z += (m * p.ldz + n) * 2;
}
inline LinearEpi epi_of(const LinearParams& p) {
    return LinearEpi{p.bias, p.R, p.Z, p.C, p.ldr, p.ldz, p.ldc, p.M, p.N, p.bias_type, p.act};
}
// f(T, OUT) for the types of a call, as integral constants.
template <class F>
hipError_t by_type(int in_type, int out_type, F&& f) {
    typedef std::integral_constant<int, DT_BF16> B;
    typedef std::integral_constant<int, DT_F16> H;
    typedef std::integral_constant<int, DT_F32> S;
    if (in_type == DT_BF16) return out_type == DT_F32 ? f(B{}, S{}) : f(B{}, B{});
    return out_type == DT_F32 ? f(H{}, S{}) : f(H{}, H{});
}

}  // namespace gemm
