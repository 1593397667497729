// rmsnorm.hip -- root-mean-square norm of rows, with the residual's addition and an output
// in 8 bits, and its backward pass.
//
//   h = x + r, rounded to its type          rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h * rstd * w                        8 bits: s = max(amax |y| / 448, 2^-126), q = rne(y / s)
//
// The norm is of the rounded h, the one that is kept: a backward pass that reads it
// differentiates the function that ran, and norming h later gives the same bits.
//
// Bytes bound it (each element is read and written once), so a row lives in registers
// between the pass that sums and the pass that writes: WPR waves share a row, each thread V
// vectors of 16 bytes of it, and rows of any pitch use unaligned vectors with only a row's
// last, partial vector element by element.  Rows longer than the registers hold are read
// once per pass by the looping kernel.
#include <algorithm>

#include "ops_common.hpp"

namespace gemm {
namespace {

constexpr float kF8Max = 448.0f;
constexpr float kTiny = 1.17549435e-38f;  // smallest normal: the scale of a row of zeros, whose reciprocal is finite

// Vector of row elements c .. c+VE-1; elements at or past `cols` are 0 and not read.
template <int T>
__device__ __forceinline__ u32x4 load_vec(const char* row, int c, int cols) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE;
    if (c + VE <= cols) return load16(row + (int64_t)c * SZ);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if (c + e < cols) {
            if constexpr (T == DT_F32) v[e] = reinterpret_cast<const uint32_t*>(row)[c + e];
            else v[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[c + e] << ((e & 1) * 16);
        }
    return v;
}
template <int T>
__device__ __forceinline__ void store_vec(char* row, int c, int cols, const u32x4& v) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE;
    if (c + VE <= cols) { store16(row + (int64_t)c * SZ, v); return; }
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if (c + e < cols) {
            if constexpr (T == DT_F32) reinterpret_cast<uint32_t*>(row)[c + e] = v[e];
            else reinterpret_cast<uint16_t*>(row)[c + e] = (uint16_t)(v[e >> 1] >> ((e & 1) * 16));
        }
}

// VE weights from element c, as floats (ones where w is NULL, 0 past the end).
template <int VE>
__device__ __forceinline__ void load_weights(const char* w, int w_type, int c, int cols, float* f) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = 1.0f;
        return;
    }
    if (c + VE <= cols) {
        if (w_type == DT_F32) {
#pragma unroll
            for (int q = 0; q < VE / 4; ++q) {
                const u32x4 v = load16(w + ((int64_t)c + 4 * q) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[4 * q + e] = __uint_as_float(v[e]);
            }
        } else {
            uint32_t v[VE / 2];
            __builtin_memcpy(v, w + (int64_t)c * 2, VE * 2);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const uint16_t b = (uint16_t)(v[e >> 1] >> ((e & 1) * 16));
                f[e] = w_type == DT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = c + e < cols ? load_elem(w, w_type, c + e) : 0.0f;
}

// VE results from element c of an output row of type y_type.
template <int VE>
__device__ __forceinline__ void store_y(char* row, int y_type, int c, int cols, const float* f) {
    if (c + VE <= cols) {
        if (y_type == DT_F32) {
#pragma unroll
            for (int q = 0; q < VE / 4; ++q) store16(row + ((int64_t)c + 4 * q) * 4, Elem<DT_F32>::pack(f + 4 * q));
        } else if (y_type == DT_F8E4M3) {
            uint32_t v[VE / 4];
#pragma unroll
            for (int q = 0; q < VE / 4; ++q) v[q] = pack_f8x4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
            __builtin_memcpy(row + c, v, VE);
        } else {
            uint32_t v[VE / 2];
#pragma unroll
            for (int q = 0; q < VE / 2; ++q)
                v[q] = y_type == DT_BF16
                           ? (uint32_t)f32_to_bf16_bits(f[2 * q]) | ((uint32_t)f32_to_bf16_bits(f[2 * q + 1]) << 16)
                           : (uint32_t)f32_to_f16_bits(f[2 * q]) | ((uint32_t)f32_to_f16_bits(f[2 * q + 1]) << 16);
            __builtin_memcpy(row + (int64_t)c * 2, v, VE * 2);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if (c + e < cols) {
            if (y_type == DT_F32) reinterpret_cast<float*>(row)[c + e] = f[e];
            else if (y_type == DT_F8E4M3) reinterpret_cast<uint8_t*>(row)[c + e] = (uint8_t)pack_f8x4(f[e], 0.f, 0.f, 0.f);
            else reinterpret_cast<uint16_t*>(row)[c + e] = y_type == DT_BF16 ? f32_to_bf16_bits(f[e]) : f32_to_f16_bits(f[e]);
        }
}
__device__ __forceinline__ int y_size(int t) { return t == DT_F32 ? 4 : t == DT_F8E4M3 ? 1 : 2; }

// Joins a value per wave over the WPR waves of a row.  `slot`: WPR words of LDS per row
// group, free when every wave arrives here.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
    v = wave_sum(v);
    if constexpr (WPR == 1) return v;
    if (lane_id() == 0) slot[wave_id() % WPR] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) s += slot[i];
    return s;
}
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* slot) {
    v = wave_max(v);
    if constexpr (WPR == 1) return v;
    if (lane_id() == 0) slot[wave_id() % WPR] = v;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int i = 0; i < WPR; ++i) s = slot[i] > s ? slot[i] : s;
    return s;
}

// The largest |y| of a row as bits: unsigned order is the order of magnitudes, and a NaN
// is above infinity, so it reaches the scale.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    const float s = __uint_as_float(amax_bits) / kF8Max;
    return s < kTiny ? kTiny : s;   // (a NaN compares false and stays)
}
// y / s by s's reciprocal and what its product leaves, rounded as a division is: two operations more than the product
// alone, which bytes hide.  (An infinite scale has no finite values in its row.)
__device__ __forceinline__ float over_scale(float y, float s, float inv) {
    const float q = y * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, s, y), inv, q);
}

// h = x + r in T; x alone where there is no residual.
template <int T>
__device__ __forceinline__ u32x4 add_residual(const u32x4& x, const u32x4& r) {
    float f[Elem<T>::VE];
#pragma unroll
    for (int e = 0; e < Elem<T>::VE; ++e) f[e] = Elem<T>::get(x, e) + Elem<T>::get(r, e);
    return Elem<T>::pack(f);
}

// V vectors of weights from element c on, TPR vectors apart, as they lie in memory (WT: T or DT_F32); `c` of a vector
// past the end is its row's last.
template <int T, int WT>
struct Weights {
    static constexpr int VE = Elem<T>::VE, N = WT == T ? 1 : 2;   // 16-byte loads for VE weights
    u32x4 raw[N];
    __device__ __forceinline__ void load(const char* w, int c) {
        if (!w) return;
#pragma unroll
        for (int q = 0; q < N; ++q) raw[q] = load16(w + (int64_t)c * (WT == DT_F32 ? 4 : 2) + 16 * q);
    }
    __device__ __forceinline__ float get(bool ones, int e) const {
        return ones ? 1.0f : Elem<WT>::get(raw[e / Elem<WT>::VE], e % Elem<WT>::VE);
    }
};

// WPR waves per row, RPG rows per workgroup of 64*WPR*RPG threads; rows of VE elements at least.
//
// No load stands behind a branch: a vector past the row's end, or across it, is the row's last VE elements,
// and what other threads have of it is left out of the sums (and stored twice, as the same
// value; every load of a row comes before its first store).  The weights stay in registers over the rows
// of a workgroup; y is computed once for its largest magnitude and once more to be written, which
// holds fewer registers than keeping it (16384 x 8192 bf16 with residual to 8 bits: 353 -> 176 us, 5.3 TB/s; 2049 x 4001
// f16 8.6 us, 3.8 TB/s: rows that start anywhere).
template <int T, bool F8, int WT, int WPR, int RPG, int V>
__global__ __launch_bounds__(64 * WPR * RPG) void norm_kernel(const NormParams p) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE, TPR = 64 * WPR;
    static_assert(WPR == 1 || RPG == 1, "rows that share a workgroup have a wave each: no barrier in their loop");
    __shared__ float sums[2][WPR], wide[2][WPR];
    __shared__ uint32_t maxs[2][WPR];
    const int t = threadIdx.x % TPR;
    auto own = [&](int i) { return (t + i * TPR) * VE; };                 // this thread's elements ...
    auto from = [&](int i) { return min(own(i), p.cols - VE); };          // ... and where it reads them
    auto whole = [&](int i) { return (i + 1) * TPR * VE <= p.cols; };     // every thread has all of its vector
    const bool ones = p.w == nullptr;
    Weights<T, WT> w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i].load(p.w, from(i));
    // the next row is on its way while this one is summed and written (but for sixteen waves a row, which fill the registers)
    constexpr bool AHEAD = WPR < 16;
    u32x4 nx[V], nr[V];
    auto load = [&](int64_t row) {
        const char* xr = p.x + row * p.ldx * SZ;
#pragma unroll
        for (int i = 0; i < V; ++i) nx[i] = load16(xr + (int64_t)from(i) * SZ);
        if (p.r) {
            const char* rr = p.r + row * p.ldr * SZ;
#pragma unroll
            for (int i = 0; i < V; ++i) nr[i] = load16(rr + (int64_t)from(i) * SZ);
        }
    };
    int turn = 0;   // the LDS words alternate, so a row's writes never meet the previous row's reads
    int64_t row = (int64_t)blockIdx.x * RPG + threadIdx.x / TPR;
    const int64_t stride = (int64_t)gridDim.x * RPG;
    if (AHEAD && row < p.rows) load(row);
    for (; row < p.rows; row += stride) {
        if (!AHEAD) load(row);
        u32x4 v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = p.r ? add_residual<T>(nx[i], nr[i]) : nx[i];
        if (AHEAD && row + stride < p.rows) load(row + stride);
        auto squares = [&](float by) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int first = whole(i) ? 0 : own(i) - from(i);   // elements before it are other threads'
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float f = e >= first ? by * Elem<T>::get(v[i], e) : 0.0f;
                    sum = __builtin_fmaf(f, f, sum);
                }
            }
            return sum;
        };
        const float rstd = row_rstd(row_sum<WPR>(squares(1.0f), sums[turn]), p.cols, p.eps,
                                    [&](float by) { return row_sum<WPR>(squares(by), wide[turn]); });
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        if (p.h) {
            char* hr = p.h + row * p.ldh * SZ;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (own(i) < p.cols) store16(hr + (int64_t)from(i) * SZ, v[i]);
        }
        auto y = [&](int i, int e) { return w[i].get(ones, e) * (Elem<T>::get(v[i], e) * rstd); };
        float scale = 1.0f, inv = 1.0f;
        if constexpr (F8) {
            uint32_t amax = 0;   // (what is read twice is in the row anyway)
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const uint32_t b = __float_as_uint(y(i, e)) & 0x7fffffffu;
                    amax = b > amax ? b : amax;
                }
            scale = row_scale(row_max<WPR>(amax, maxs[turn]));
            inv = 1.0f / scale;
            if (t == 0) p.scale[row] = scale;
        }
        const int yt = F8 ? (int)DT_F8E4M3 : p.y_type;
        char* yr = p.y + row * p.ldy * y_size(yt);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (own(i) < p.cols) {
                float f[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) f[e] = F8 ? over_scale(y(i, e), scale, inv) : y(i, e);
                store_y<VE>(yr, yt, from(i), p.cols, f);
            }
        turn ^= 1;
    }
}

// Rows of any length: a workgroup of 16 waves reads its row once for the sum, for 8 bits
// once more for the largest magnitude, and once to write.  Every element is read and written by
// the same thread, its write after its last read, so h or y may lie on x or r.
constexpr int kLoopThreads = 1024;
template <int T>
__global__ __launch_bounds__(kLoopThreads) void norm_loop_kernel(const NormParams p) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE, W = kLoopThreads / 64;
    __shared__ float sums[2][W], wide[2][W];
    __shared__ uint32_t maxs[2][W];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const char* xr = p.x + row * p.ldx * SZ;
        const char* rr = p.r + row * p.ldr * SZ;
        auto at = [&](int c) {
            u32x4 v = load_vec<T>(xr, c, p.cols);
            if (p.r) v = add_residual<T>(v, load_vec<T>(rr, c, p.cols));
            return v;
        };
        auto squares = [&](float by) {
            float sum = 0.0f;
            for (int64_t c = (int64_t)threadIdx.x * VE; c < p.cols; c += kLoopThreads * VE) {
                const u32x4 v = at((int)c);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float f = by * Elem<T>::get(v, e);
                    sum = __builtin_fmaf(f, f, sum);
                }
            }
            return sum;
        };
        const float rstd = row_rstd(row_sum<W>(squares(1.0f), sums[turn]), p.cols, p.eps,
                                    [&](float by) { return row_sum<W>(squares(by), wide[turn]); });
        if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
        float scale = 1.0f, inv = 1.0f;
        if (p.y_type == DT_F8E4M3) {
            uint32_t amax = 0;
            for (int64_t c = (int64_t)threadIdx.x * VE; c < p.cols; c += kLoopThreads * VE) {
                const u32x4 v = at((int)c);
                float f[VE];
                load_weights<VE>(p.w, p.w_type, (int)c, p.cols, f);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const uint32_t b = __float_as_uint(f[e] * (Elem<T>::get(v, e) * rstd)) & 0x7fffffffu;
                    if (c + e < p.cols) amax = b > amax ? b : amax;
                }
            }
            scale = row_scale(row_max<W>(amax, maxs[turn]));
            inv = 1.0f / scale;
            if (threadIdx.x == 0) p.scale[row] = scale;
        }
        char* yr = p.y + row * p.ldy * y_size(p.y_type);
        for (int64_t c = (int64_t)threadIdx.x * VE; c < p.cols; c += kLoopThreads * VE) {
            const u32x4 v = at((int)c);
            float f[VE];
            load_weights<VE>(p.w, p.w_type, (int)c, p.cols, f);
#pragma unroll
            for (int e = 0; e < VE; ++e) f[e] *= Elem<T>::get(v, e) * rstd;
            if (p.y_type == DT_F8E4M3) {
#pragma unroll
                for (int e = 0; e < VE; ++e) f[e] = over_scale(f[e], scale, inv);
            }
            if (p.h) store_vec<T>(p.h + row * p.ldh * SZ, (int)c, p.cols, v);
            store_y<VE>(yr, p.y_type, (int)c, p.cols, f);
        }
        turn ^= 1;
    }
}

constexpr int64_t kMaxGrid = 1 << 20;   // workgroups of a launch; more rows loop

// As many workgroups as the registers let stay on the card; each takes every so many rows.
template <int T, bool F8, int WT, int WPR, int RPG, int V>
hipError_t go(const NormParams& p, hipStream_t st) {
    int64_t grid = (p.rows + RPG - 1) / RPG;
    const int64_t most = (int64_t)num_compute_units() * (V == 1 ? 8 : 4);
    if (grid > most) grid = most;
    hipLaunchKernelGGL((norm_kernel<T, F8, WT, WPR, RPG, V>), dim3((unsigned)grid), dim3(64 * WPR * RPG), 0, st, p);
    return hipGetLastError();
}

template <int T, bool F8, int WT>
hipError_t norm_of(const NormParams& p, hipStream_t st) {
    const int64_t vecs = ((int64_t)p.cols + Elem<T>::VE - 1) / Elem<T>::VE;
    if (p.cols >= Elem<T>::VE) {
        if (vecs <= 64) return go<T, F8, WT, 1, 4, 1>(p, st);
        if (vecs <= 128) return go<T, F8, WT, 1, 4, 2>(p, st);
        if (vecs <= 256) return go<T, F8, WT, 4, 1, 1>(p, st);
        if (vecs <= 512) return go<T, F8, WT, 4, 1, 2>(p, st);
        if (vecs <= 1024) return go<T, F8, WT, 4, 1, 4>(p, st);
        if (vecs <= 2048) return go<T, F8, WT, 8, 1, 4>(p, st);
        if (vecs <= 4096) return go<T, F8, WT, 16, 1, 4>(p, st);
    }
    hipLaunchKernelGGL((norm_loop_kernel<T>), dim3((unsigned)(p.rows > kMaxGrid ? kMaxGrid : p.rows)),
                       dim3(kLoopThreads), 0, st, p);
    return hipGetLastError();
}
template <int T>
hipError_t norm_in(const NormParams& p, hipStream_t st) {
    const bool f8 = p.y_type == DT_F8E4M3;
    if constexpr (T != DT_F32) {
        if (p.w && p.w_type == DT_F32) return f8 ? norm_of<T, true, DT_F32>(p, st) : norm_of<T, false, DT_F32>(p, st);
    }
    return f8 ? norm_of<T, true, T>(p, st) : norm_of<T, false, T>(p, st);
}

}  // namespace

hipError_t launch_norm(int in_type, const NormParams& p, hipStream_t st) {
    switch (in_type) {
        case DT_F32: return norm_in<DT_F32>(p, st);
        case DT_BF16: return norm_in<DT_BF16>(p, st);
        case DT_F16: return norm_in<DT_F16>(p, st);
    }
    return hipErrorInvalidValue;
}

// ==================================================================== backward
//   g = dy * w, u = h * rstd:   dx = rstd * (g - u * mean(g * u)) + dh,   dw = sum over rows of dy * u
//
// One pass: a workgroup takes the rows b, b + parts, ... (b its index); a row's dy and h stay
// in registers between the sum and dx, and dy * u is added into the thread's own columns of
// dw.  The partial rows of dw, one per workgroup, are joined by a second launch in a fixed
// order, so the result is the same on every run.
//
// Few rows are over before the second launch begins.  There the workgroups keep no dw, and waves of the same launch
// sum it, 64 bytes of all rows each: dw needs no row's mean.  They read dy and h a second time, out of a cache, and
// before or after dx is written, so dx lies on neither; and they add in the order of the two launches, which such a dx takes.
namespace {

constexpr int kJoinSlices = 16;   // of dw's partial rows, each summed in order, then joined in order

// dw of the 64 bytes of columns that strip b has: four lanes side by side, a slice of the rows each sixteen lanes.
template <int T, int RPG>
__device__ __forceinline__ void norm_bwd_strip(const NormBwdParams& p, int b) {
#pragma clang fp contract(off)
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE;
    const int lane = (int)threadIdx.x % 64, own = (b * 4 + lane % 4) * VE, from = min(own, p.cols - VE);
    const char* dy0 = p.dy + (int64_t)from * SZ;
    const char* h0 = p.h + (int64_t)from * SZ;
    float sum[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) sum[e] = 0.0f;
    const int rows = (int)p.rows, groups = (rows + RPG - 1) / RPG;
#pragma unroll 8 / RPG
    for (int g = lane / 4; g < groups; g += kJoinSlices) {
        float part[VE];
#pragma unroll
        for (int i = 0; i < RPG; ++i) {
            const int64_t row = min(g * RPG + i, rows - 1);
            const u32x4 dy = load16(dy0 + row * p.lddy * SZ), h = load16(h0 + row * p.ldh * SZ);
            const float rstd = p.rstd[row];
            const bool there = g * RPG + i < rows;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float u = Elem<T>::get(h, e) * rstd, du = Elem<T>::get(dy, e) * u;
                part[e] = i == 0 ? du : there ? part[e] + du : part[e];
            }
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) sum[e] += part[e];
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        float all = __shfl(sum[e], lane % 4, 64);
#pragma unroll
        for (int q = 1; q < kJoinSlices; ++q) all += __shfl(sum[e], q * 4 + lane % 4, 64);
        if (lane < 4 && from + e >= own) p.dw[from + e] = all;
    }
}

// Vectors past or across a row's end are read as in norm_kernel.
template <int T, int WT, int WPR, int RPG, int V>
__global__ __launch_bounds__(64 * WPR * RPG) void norm_bwd_kernel(const NormBwdParams p) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE, TPR = 64 * WPR;
    static_assert(WPR == 1 || RPG == 1, "rows that share a workgroup have a wave each: no barrier in their loop");
    __shared__ float sums[2][WPR];
    __shared__ float join[RPG > 1 ? (RPG - 1) * TPR * V * VE : 1];
    const int strips = p.strip_blocks, blocks = (int)gridDim.x - strips;
    if ((int)blockIdx.x < strips) {
        const int strip = (int)blockIdx.x * WPR * RPG + (int)threadIdx.x / 64;
        if (strip * 4 * VE < p.cols) norm_bwd_strip<T, RPG>(p, strip);
        return;
    }
    const int t = threadIdx.x % TPR;
    auto own = [&](int i) { return (t + i * TPR) * VE; };
    auto from = [&](int i) { return min(own(i), p.cols - VE); };
    auto whole = [&](int i) { return (i + 1) * TPR * VE <= p.cols; };
    const bool ones = p.w == nullptr;
    float acc[V][VE];
    Weights<T, WT> w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        w[i].load(p.w, from(i));
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[i][e] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = (int64_t)((int)blockIdx.x - strips) * RPG + threadIdx.x / TPR; row < p.rows; row += (int64_t)blocks * RPG) {
        u32x4 dy[V], h[V], dh[V];
        const char* yr = p.dy + row * p.lddy * SZ;
        const char* hr = p.h + row * p.ldh * SZ;
#pragma unroll
        for (int i = 0; i < V; ++i) dy[i] = load16(yr + (int64_t)from(i) * SZ);
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = load16(hr + (int64_t)from(i) * SZ);
        if (p.dh) {
            const char* dr = p.dh + row * p.lddh * SZ;
#pragma unroll
            for (int i = 0; i < V; ++i) dh[i] = load16(dr + (int64_t)from(i) * SZ);
        }
        const float rstd = p.rstd[row];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int first = whole(i) ? 0 : own(i) - from(i);   // elements before it are other threads'
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float du = e >= first ? Elem<T>::get(dy[i], e) * (Elem<T>::get(h[i], e) * rstd) : 0.0f;
                acc[i][e] += du;
                sum = __builtin_fmaf(du, w[i].get(ones, e), sum);
            }
        }
        // dx may lie on dh, and a row's last elements may be another wave's to store as well: dh is here before the barrier in
        // row_sum(), as dy and h are, which the sum has used.  (A wait, as uses of dh's registers here would make fp32 rows of
        // 9000 and more spill: 2000 x 12000 116 us instead of 85.)
        if (WPR > 1 && p.dh) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const float mean = row_sum<WPR>(sum, sums[turn]) / (float)p.cols;
        char* xr = p.dx + row * p.lddx * SZ;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (own(i) < p.cols) {
                float f[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    f[e] = rstd * (Elem<T>::get(dy[i], e) * w[i].get(ones, e) - Elem<T>::get(h[i], e) * rstd * mean);
                    if (p.dh) f[e] += Elem<T>::get(dh[i], e);
                }
                store16(xr + (int64_t)from(i) * SZ, Elem<T>::pack(f));
            }
        turn ^= 1;
    }
    if (!p.dw || strips) return;
    if constexpr (RPG > 1) {
        // the waves' sums meet in wave order in the first one
        const int g = threadIdx.x / TPR;
        if (g > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) join[((g - 1) * V * VE + i * VE + e) * TPR + t] = acc[i][e];
        }
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int q = 0; q < RPG - 1; ++q)
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) acc[i][e] += join[(q * V * VE + i * VE + e) * TPR + t];
    }
    float* out = gridDim.x == 1 ? p.dw : p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (own(i) + VE <= p.cols) {
            store_y<VE>(reinterpret_cast<char*>(out), DT_F32, own(i), p.cols, acc[i]);
        } else {   // what this thread alone has of the row's last vector
            const int first = own(i) - from(i);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (e >= first) out[from(i) + e] = acc[i][e];
        }
    }
}

// dx for rows of any length: the row is read twice.
template <int T>
__global__ __launch_bounds__(kLoopThreads) void norm_bwd_loop_kernel(const NormBwdParams p) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE, W = kLoopThreads / 64;
    __shared__ float sums[2][W];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const char* yr = p.dy + row * p.lddy * SZ;
        const char* hr = p.h + row * p.ldh * SZ;
        const char* dr = p.dh + row * p.lddh * SZ;
        char* xr = p.dx + row * p.lddx * SZ;
        const float rstd = p.rstd[row];
        float sum = 0.0f;
        for (int64_t c = (int64_t)threadIdx.x * VE; c < p.cols; c += kLoopThreads * VE) {
            const u32x4 dy = load_vec<T>(yr, (int)c, p.cols), h = load_vec<T>(hr, (int)c, p.cols);
            float w[VE];
            load_weights<VE>(p.w, p.w_type, (int)c, p.cols, w);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                sum = __builtin_fmaf(Elem<T>::get(dy, e) * (Elem<T>::get(h, e) * rstd), w[e], sum);
        }
        const float mean = row_sum<W>(sum, sums[turn]) / (float)p.cols;
        for (int64_t c = (int64_t)threadIdx.x * VE; c < p.cols; c += kLoopThreads * VE) {
            const u32x4 dy = load_vec<T>(yr, (int)c, p.cols), h = load_vec<T>(hr, (int)c, p.cols);
            u32x4 dh = {0u, 0u, 0u, 0u};
            if (p.dh) dh = load_vec<T>(dr, (int)c, p.cols);
            float w[VE], f[VE];
            load_weights<VE>(p.w, p.w_type, (int)c, p.cols, w);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float u = Elem<T>::get(h, e) * rstd;
                f[e] = rstd * (Elem<T>::get(dy, e) * w[e] - u * mean);
                if (p.dh) f[e] += Elem<T>::get(dh, e);
            }
            store_vec<T>(xr, (int)c, p.cols, Elem<T>::pack(f));
        }
        turn ^= 1;
    }
}

// Partial rows of dw for rows of any length: a thread per column, workgroup (x, b) the rows
// b, b + parts, ...  Runs before dx is written, which may lie on dy or h.
template <int T>
__global__ __launch_bounds__(256) void norm_bwd_dw_kernel(const NormBwdParams p) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float sum = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y)
        sum = __builtin_fmaf(load_elem(p.dy, T, row * p.lddy + c), load_elem(p.h, T, row * p.ldh + c) * p.rstd[row], sum);
    (gridDim.y == 1 ? p.dw : p.part + (int64_t)blockIdx.y * p.cols)[c] = sum;
}

// dw = the sum of the partial rows: 64 columns per workgroup, 16 slices of the rows, each
// summed in order and the slices joined in order.
__global__ __launch_bounds__(64 * kJoinSlices) void norm_bwd_join_kernel(const float* part, float* dw, int cols, int parts) {
    __shared__ float s[kJoinSlices][64];
    const int lane = threadIdx.x % 64, q = threadIdx.x / 64;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float sum = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int r = q; r < parts; r += kJoinSlices) sum += part[(int64_t)r * cols + c];
    }
    s[q][lane] = sum;
    __syncthreads();
    if (q > 0 || c >= cols) return;
#pragma unroll
    for (int i = 1; i < kJoinSlices; ++i) sum += s[i][lane];
    dw[c] = sum;
}

__global__ __launch_bounds__(256) void zero_kernel(float* p, int n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

template <int T, int WT, int WPR, int RPG, int V>
hipError_t go_bwd(const NormBwdParams& p, hipStream_t st) {
    if (p.strip_blocks) {
        NormBwdParams q = p;
        const int strips = (p.cols + 4 * Elem<T>::VE - 1) / (4 * Elem<T>::VE);
        q.strip_blocks = (strips + WPR * RPG - 1) / (WPR * RPG);
        const unsigned blocks = (unsigned)((p.rows + RPG - 1) / RPG);
        hipLaunchKernelGGL((norm_bwd_kernel<T, WT, WPR, RPG, V>), dim3(q.strip_blocks + blocks), dim3(64 * WPR * RPG), 0, st, q);
    } else {
        hipLaunchKernelGGL((norm_bwd_kernel<T, WT, WPR, RPG, V>), dim3(p.parts), dim3(64 * WPR * RPG), 0, st, p);
    }
    return hipGetLastError();
}
// Vectors of 16 bytes that the registers hold of a row (fp32 has half the sums of dw to keep).
template <int T>
constexpr int64_t kBwdVecs = T == DT_F32 ? 4096 : 2048;

template <int T, int WT>
hipError_t bwd_rows(const NormBwdParams& p, int64_t vecs, hipStream_t st) {
    if (vecs <= 64) return go_bwd<T, WT, 1, 4, 1>(p, st);
    if (vecs <= 128) return go_bwd<T, WT, 1, 4, 2>(p, st);
    if (vecs <= 256) return go_bwd<T, WT, 4, 1, 1>(p, st);
    if (vecs <= 512) return go_bwd<T, WT, 4, 1, 2>(p, st);
    if (vecs <= 1024) return go_bwd<T, WT, 8, 1, 2>(p, st);
    if constexpr (T == DT_F32) {
        if (vecs > 2048) return go_bwd<T, WT, 16, 1, 4>(p, st);
    }
    return go_bwd<T, WT, 16, 1, 2>(p, st);
}

// Whether dx lies apart from what the strips read.
template <int T>
bool apart(const NormBwdParams& p) {
    auto end = [&](const char* at, int64_t ld) { return at + ((p.rows - 1) * ld + p.cols) * Elem<T>::SIZE; };
    auto clear = [&](const char* at, int64_t ld) { return end(at, ld) <= p.dx || end(p.dx, p.lddx) <= at; };
    return clear(p.dy, p.lddy) && clear(p.h, p.ldh);
}
// 40 x 4096 bf16 6.2 us with a second launch, 4.1 so; 100 rows 7.6 and 5.3; 256 rows 9.2 and 10.6.
constexpr int64_t kStripRows = 128;

template <int T>
hipError_t bwd_of(const NormBwdParams& f, hipStream_t st) {
    NormBwdParams p = f;
    p.strip_blocks = p.dw && p.parts > 1 && p.rows <= kStripRows && apart<T>(p);
    if (p.rows == 0) {  // dw is a sum of nothing
        hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(((int64_t)p.cols + 255) / 256)), dim3(256), 0, st, p.dw, p.cols);
        return hipGetLastError();
    }
    const int64_t vecs = ((int64_t)p.cols + Elem<T>::VE - 1) / Elem<T>::VE;
    hipError_t e;
    const bool strips = p.strip_blocks && p.cols >= Elem<T>::VE && vecs <= kBwdVecs<T>;
    if (p.cols >= Elem<T>::VE && vecs <= kBwdVecs<T>) {
        if (p.w && p.w_type == DT_F32) e = bwd_rows<T, DT_F32>(p, vecs, st);
        else e = bwd_rows<T, T>(p, vecs, st);
    }
    else {
        e = hipSuccess;
        if (p.dw) {
            hipLaunchKernelGGL((norm_bwd_dw_kernel<T>), dim3((unsigned)(((int64_t)p.cols + 255) / 256), p.parts),
                               dim3(256), 0, st, p);
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((norm_bwd_loop_kernel<T>), dim3((unsigned)(p.rows > kMaxGrid ? kMaxGrid : p.rows)),
                           dim3(kLoopThreads), 0, st, p);
        e = hipGetLastError();
    }
    if (e != hipSuccess || !p.dw || p.parts == 1 || strips) return e;
    hipLaunchKernelGGL(norm_bwd_join_kernel, dim3((unsigned)(((int64_t)p.cols + 63) / 64)), dim3(64 * kJoinSlices), 0, st,
                       p.part, p.dw, p.cols, p.parts);
    return hipGetLastError();
}

}  // namespace

int norm_bwd_parts(int in_type, int64_t rows, int cols) {
    const int ve = in_type == DT_F32 ? 4 : 8;
    const int64_t vecs = ((int64_t)cols + ve - 1) / ve;
    if (cols < ve || vecs > (in_type == DT_F32 ? kBwdVecs<DT_F32> : kBwdVecs<DT_BF16>))   // looping kernels: slices of the rows
        return (int)(rows < 64 ? (rows < 1 ? 1 : rows) : 64);
    const int per = vecs <= 128 ? 4 : 1;
    const int64_t groups = (rows + per - 1) / per;
    // Three rows in turn cost less than the launch that joins; many rows are shared by two at least, as a partial row of dw
    // costs half a row of the pass (513 x 3001 fp32: 256 parts 9.8 us, 512 parts 11.4).
    const int64_t most = 512, parts = groups <= 3 ? 1 : groups <= 256 ? groups : std::max<int64_t>(256, groups / 2);
    return (int)(parts < most ? parts : most);
}

hipError_t launch_norm_bwd(int in_type, const NormBwdParams& p, hipStream_t st) {
    switch (in_type) {
        case DT_F32: return bwd_of<DT_F32>(p, st);
        case DT_BF16: return bwd_of<DT_BF16>(p, st);
        case DT_F16: return bwd_of<DT_F16>(p, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace gemm
