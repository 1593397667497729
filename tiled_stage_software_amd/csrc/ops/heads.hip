// heads.hip -- root-mean-square norm of each head of the queries and keys with the rotation by position, and its
// backward pass.
//
//   u = x / sqrt(mean(x^2) + eps),  v = u * w,  y = v with its first rot elements turned in pairs:
//   (y_i, y_j) = (v_i c - v_j s, v_j c + v_i s), c and s from the table's row of the token's position
//   g = dy turned back:  dw = sum over tokens and heads of g u,  dx = rstd (g w - u mean(g w u))
//
// In fp32 from the elements to the one rounding of y (dx).  A wave has a row (a head of a token) at a time in its registers, a
// lane every 64th element; partners of a pair meet in LDS that belongs to the wave, so any head size, rotated
// part and pairing runs the same way.  A position outside the table turns by NaN: nothing is read there, and it shows.
#include <algorithm>

#include "ops_common.hpp"

namespace gemm {
namespace {

constexpr int kWaves = 4;

template <int T>
__device__ __forceinline__ float load1(const char* p, int64_t i) {
    if constexpr (T == DT_F32) return reinterpret_cast<const float*>(p)[i];
    else return to_f32<T>(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <int T>
__device__ __forceinline__ void store1(char* p, int64_t i, float v) {
    if constexpr (T == DT_F32) reinterpret_cast<float*>(p)[i] = v;
    else reinterpret_cast<uint16_t*>(p)[i] = from_f32<T>(v);
}
__device__ __forceinline__ int64_t at(const HeadsTensor& t, int64_t token, int head) { return token * t.ld + head * t.hs; }

// The other element of e's pair, and e's place in the table's row; the first of a pair has the smaller index.
struct Pair {
    int other, col;
    bool first;
};
__device__ __forceinline__ Pair pair_of(const HeadsParams& p, int e) {
    if (p.neighbours) return Pair{e ^ 1, e >> 1, (e & 1) == 0};
    const int half = p.rot / 2;
    return e < half ? Pair{e + half, e, true} : Pair{e - half, e - half, false};
}
// cos and sin of a token at the table's column.
__device__ __forceinline__ void angle(const HeadsParams& p, int64_t pos, int col, float& c, float& s) {
    if (pos < 0 || pos >= p.table) {
        c = s = __builtin_nanf("");
        return;
    }
    c = p.cos[pos * p.ldt + col];
    s = p.sin[pos * p.ldt + col];
}

// NE elements a lane: heads of up to 64 * NE.
template <int T, int NE>
__global__ __launch_bounds__(64 * kWaves) void heads_kernel(const HeadsParams p) {
    __shared__ float rows[kWaves][64 * NE];
    float* row = rows[wave_id()];
    const int lane = lane_id();
    const int64_t all = p.tokens * (p.heads[0] + p.heads[1]);
    for (int64_t r = (int64_t)blockIdx.x * kWaves + wave_id(); r < all; r += (int64_t)gridDim.x * kWaves) {
        const int64_t token = r / (p.heads[0] + p.heads[1]);
        int head = (int)(r % (p.heads[0] + p.heads[1]));
        const int k = head >= p.heads[0];
        head -= k ? p.heads[0] : 0;
        const int64_t pos = p.rot ? p.pos[token] : 0;
        float v[NE], sum = 0.0f;
        const int64_t from = at(p.x[k], token, head);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            v[i] = e < p.dim ? load1<T>(p.x[k].p, from + e) : 0.0f;
            sum = __builtin_fmaf(v[i], v[i], sum);
        }
        const float rstd = row_rstd(wave_sum(sum), p.dim, p.eps, [&](float by) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) s = __builtin_fmaf(v[i] * by, v[i] * by, s);
            return wave_sum(s);
        });
        wave_fence();
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            if (e >= p.dim) continue;
            v[i] *= rstd;
            if (p.w[k]) v[i] *= load_elem(p.w[k], p.w_type, e);
            row[e] = v[i];
        }
        wave_fence();
        char* out = const_cast<char*>(p.y[k].p);
        const int64_t to = at(p.y[k], token, head);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            if (e >= p.dim) continue;
            float y = v[i];
            if (e < p.rot) {
                const Pair q = pair_of(p, e);
                float c, s;
                angle(p, pos, q.col, c, s);
                y = q.first ? v[i] * c - row[q.other] * s : v[i] * c + row[q.other] * s;
            }
            store1<T>(out, to + e, y);
        }
    }
}

template <int T, int NE>
__global__ __launch_bounds__(64 * kWaves) void heads_bwd_kernel(const HeadsParams p) {
    __shared__ float rows[kWaves][64 * NE];
    float* row = rows[wave_id()];
    const int lane = lane_id();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float dw[NE], w[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            dw[i] = 0.0f;
            w[i] = p.w[k] && e < p.dim ? load_elem(p.w[k], p.w_type, e) : 1.0f;
        }
        const int64_t all = p.tokens * p.heads[k];
        for (int64_t r = (int64_t)blockIdx.x * kWaves + wave_id(); r < all; r += (int64_t)gridDim.x * kWaves) {
            const int64_t token = r / p.heads[k];
            const int head = (int)(r % p.heads[k]);
            const int64_t pos = p.rot ? p.pos[token] : 0;
            float x[NE], g[NE], sum = 0.0f;
            const int64_t from = at(p.x[k], token, head), dfrom = at(p.dy[k], token, head);
            wave_fence();
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                x[i] = e < p.dim ? load1<T>(p.x[k].p, from + e) : 0.0f;
                g[i] = e < p.dim ? load1<T>(p.dy[k].p, dfrom + e) : 0.0f;
                row[e] = g[i];
                sum = __builtin_fmaf(x[i], x[i], sum);
            }
            wave_fence();
            const float rstd = row_rstd(wave_sum(sum), p.dim, p.eps, [&](float by) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NE; ++i) s = __builtin_fmaf(x[i] * by, x[i] * by, s);
                return wave_sum(s);
            });
            float through = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                if (e < p.rot) {
                    const Pair q = pair_of(p, e);
                    float c, s;
                    angle(p, pos, q.col, c, s);
                    g[i] = q.first ? g[i] * c + row[q.other] * s : g[i] * c - row[q.other] * s;
                }
                x[i] *= rstd;
                dw[i] = __builtin_fmaf(g[i], x[i], dw[i]);
                g[i] *= w[i];
                through = __builtin_fmaf(g[i], x[i], through);
            }
            through = wave_sum(through) / (float)p.dim;
            char* out = const_cast<char*>(p.y[k].p);
            const int64_t to = at(p.y[k], token, head);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                if (e < p.dim) store1<T>(out, to + e, rstd * (g[i] - x[i] * through));
            }
        }
        if (!p.dw[k]) continue;   // the same in every thread
        wave_fence();
#pragma unroll
        for (int i = 0; i < NE; ++i) row[lane + 64 * i] = dw[i];
        __syncthreads();
        float* to = p.parts > 1 ? p.part + ((int64_t)blockIdx.x * 2 + k) * p.dim : p.dw[k];
        for (int e = threadIdx.x; e < p.dim; e += 64 * kWaves) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) s += rows[q][e];
            to[e] = s;
        }
        __syncthreads();
    }
}

// dw = the parts' sums in order: 64 elements of queries' or keys' weights a workgroup, every sixteenth part a wave.
__global__ __launch_bounds__(1024) void heads_join_kernel(const HeadsParams p) {
    __shared__ float sums[16][64];
    const int k = blockIdx.y, e = (int)blockIdx.x * 64 + lane_id(), w = wave_id();
    if (!p.dw[k]) return;
    float s = 0.0f;
    if (e < p.dim) {
#pragma unroll 8
        for (int i = w; i < p.parts; i += 16) s += p.part[((int64_t)i * 2 + k) * p.dim + e];
    }
    sums[w][lane_id()] = s;
    __syncthreads();
    if (w != 0 || e >= p.dim) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sums[i][lane_id()];
    p.dw[k][e] = s;
}

template <class F>
hipError_t by_size(int type, int dim, F&& f) {
    auto sized = [&](auto t) {
        if (dim <= 64) return f(t, std::integral_constant<int, 1>{});
        if (dim <= 128) return f(t, std::integral_constant<int, 2>{});
        if (dim <= 256) return f(t, std::integral_constant<int, 4>{});
        return f(t, std::integral_constant<int, 16>{});
    };
    if (type == DT_F32) return sized(std::integral_constant<int, DT_F32>{});
    if (type == DT_BF16) return sized(std::integral_constant<int, DT_BF16>{});
    return sized(std::integral_constant<int, DT_F16>{});
}

}  // namespace

hipError_t launch_heads(int in_type, const HeadsParams& p, hipStream_t st) {
    const int64_t rows = p.tokens * (p.heads[0] + p.heads[1]);
    const int64_t grid = std::min<int64_t>((rows + kWaves - 1) / kWaves, 16 * (int64_t)num_compute_units());
    return by_size(in_type, p.dim, [&](auto t, auto n) {
        hipLaunchKernelGGL((heads_kernel<decltype(t)::value, decltype(n)::value>), dim3((unsigned)grid), dim3(64 * kWaves), 0, st, p);
        return hipGetLastError();
    });
}

int heads_bwd_parts(const HeadsParams& p) {
    const int64_t rows = p.tokens * std::max(p.heads[0], p.heads[1]);
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + kWaves - 1) / kWaves, 4 * (int64_t)num_compute_units()));
}

hipError_t launch_heads_bwd(int in_type, const HeadsParams& p, hipStream_t st) {
    const hipError_t e = by_size(in_type, p.dim, [&](auto t, auto n) {
        hipLaunchKernelGGL((heads_bwd_kernel<decltype(t)::value, decltype(n)::value>), dim3((unsigned)p.parts), dim3(64 * kWaves), 0, st, p);
        return hipGetLastError();
    });
    if (e != hipSuccess || p.parts == 1 || (!p.dw[0] && !p.dw[1])) return e;
    hipLaunchKernelGGL(heads_join_kernel, dim3((unsigned)((p.dim + 63) / 64), 2), dim3(1024), 0, st, p);
    return hipGetLastError();
}

}  // namespace gemm
