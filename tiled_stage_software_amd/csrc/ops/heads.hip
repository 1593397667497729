// heads.hip -- root-mean-square norm of each head of the queries and keys with the rotation by position, and its
// backward pass.
//
//   u = x / sqrt(mean(x^2) + eps),  v = u * w,  y = v with its first rot elements turned in pairs:
//   (y_i, y_j) = (v_i c - v_j s, v_j c + v_i s), c and s from the table's row of the token's position
//   g = dy turned back:  dw = sum over tokens and heads of g u,  dx = rstd (g w - u mean(g w u))
//
// In fp32 from the elements to the one rounding of y (dx).  Bytes bound it.  LPH lanes share a head, each with IPL items of two
// 16-byte vectors: of the part that turns in halves, a vector of the first half and its partners in the second; else two
// neighbouring vectors, which hold their pairs themselves.  So both of a pair are in one lane and nothing is exchanged but the
// sums.  A wave takes 64 / LPH heads of one token at a time, the next ones on their way, and keeps the token's cosines and sines.
// Where a part is no whole number of vectors its last vector lies over the one before, stores the same values again and
// is left out of the sums where it does; a part shorter than a vector goes element by element.  A position outside
// the table turns by NaN: nothing is read there, and it shows.
//
// Measured on bf16 of 128 elements a head, 32 + 8 heads, all turned: 16384 tokens forward 70 us (4.8 TB/s, a large copy 4.75 to
// 5.1), 8192 backward 59 us (4.3 TB/s) with the join of dw.  What held it: a lane's accesses behind branches (82 -> 71 us
// forward), arrays indexed by how pairs lie (scratch memory: 82 -> 59 us backward), positions read by vector loads, more
// workgroups than the card holds at once.  Overlapping vectors take a third more time for their bytes, short parts three times.
#include <algorithm>

#include "ops_common.hpp"

namespace gemm {
namespace {

constexpr int kWaves = 4, kEach = 4;   // waves of a workgroup; jobs of a wave, where there are enough

// What a head's parts (the one that turns, by halves or whole, and the rest) are made of.
enum : int {
    WHOLE = 0,     // whole vectors
    OVERLAP = 1,   // whole vectors, the last over the one before it
    SHORT = 2      // some part is shorter than a vector
};

// Two vectors of a head: elements at[v] .. at[v] + count[v] - 1 (VE, fewer in a short part, or none), of which this item owns
// those from first[v] on.
struct Item {
    int at[2], first[2], count[2];
    bool turns;
};
// Vector i of the part [from, to).
template <int VE>
__device__ __forceinline__ void place(Item& it, int v, int i, int from, int to) {
    const int start = from + i * VE;
    it.at[v] = start;
    it.first[v] = 0;
    it.count[v] = start < to ? min(VE, to - from) : 0;
    if (to - from >= VE && start < to && start > to - VE) {
        it.first[v] = start - (to - VE);
        it.at[v] = to - VE;
    }
}
// Items of a head: those that turn, then the others.
template <int VE>
__host__ __device__ __forceinline__ int turning_items(int rot, int neighbours) {
    const int vectors = neighbours ? (rot + VE - 1) / VE : 2 * ((rot / 2 + VE - 1) / VE);
    return (vectors + 1) / 2;
}
template <int VE>
__host__ __device__ __forceinline__ int items_of(int dim, int rot, int neighbours) {
    return turning_items<VE>(rot, neighbours) + ((dim - rot + VE - 1) / VE + 1) / 2;
}
template <int VE>
__device__ __forceinline__ Item item_of(const HeadsParams& p, int q) {
    Item it;
    const int turning = turning_items<VE>(p.rot, p.neighbours);
    it.turns = q < turning;
    if (it.turns && !p.neighbours) {
        place<VE>(it, 0, q, 0, p.rot / 2);
        place<VE>(it, 1, q, p.rot / 2, p.rot);
    } else {
        const int from = it.turns ? 0 : p.rot, to = it.turns ? p.rot : p.dim, i = 2 * (it.turns ? q : q - turning);
        place<VE>(it, 0, i, from, to);
        place<VE>(it, 1, i + 1, from, to);
    }
    return it;
}

// Memory from `base` on, for loads and stores by 32-bit offsets: past kReach nothing is read (zeros come) or written.  So lanes that
// have nothing take part in every access, and none stands behind a branch, behind which a wait for a load would wait for
// the stores of the step before too.
constexpr uint32_t kReach = 0x7fffffffu, kNowhere = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t reach(const char* base, bool there = true) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, there ? (int)kReach : 0, 0x00020000);
}

// An item's elements in pairs (a, b) in fp32: (e, e) of its two vectors where pairs lie in halves, else neighbours, vector
// by vector.  Items that do not turn are held the same way.
template <int VE>
struct Pairs {
    float a[VE], b[VE];
};
// f(pair, element of vector 0, or of the pair's vector; element of vector 1, or the next one; the vectors' numbers) of each pair.
template <int VE, class F>
__device__ __forceinline__ void each_pair(bool halves, F&& f) {
    if (halves) {
#pragma unroll
        for (int e = 0; e < VE; ++e) f(e, 0, e, 1, e);
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) f(e, e / (VE / 2), 2 * (e % (VE / 2)), e / (VE / 2), 2 * (e % (VE / 2)) + 1);
    }
}

// An item's two vectors as they lie in memory, zeros where it has none.
template <int T, int SHAPE>
struct Vec {
    static constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE;
    u32x4 raw[2];
    // head: offset of the lane's head from `base`.
    __device__ __forceinline__ void load(const char* base, uint32_t head, bool there, const Item& it) {
        const __amdgpu_buffer_rsrc_t rs = reach(base);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const bool whole = there && (SHAPE != SHORT ? it.count[v] > 0 : it.count[v] == VE);
            raw[v] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, whole ? head + it.at[v] * SZ : kNowhere, 0, 0));
            if constexpr (SHAPE == SHORT) {
                if (there && !whole) {
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        if (e < it.count[v]) {
                            if constexpr (T == DT_F32) raw[v][e] = reinterpret_cast<const uint32_t*>(base + head)[it.at[v] + e];
                            else raw[v][e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(base + head)[it.at[v] + e] << ((e & 1) * 16);
                        }
                }
            }
        }
    }
    __device__ __forceinline__ void store(char* base, uint32_t head, bool there, const Item& it) const {
        const __amdgpu_buffer_rsrc_t rs = reach(base);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const bool whole = there && (SHAPE != SHORT ? it.count[v] > 0 : it.count[v] == VE);
            __builtin_amdgcn_raw_buffer_store_b128(raw[v], rs, whole ? head + it.at[v] * SZ : kNowhere, 0, 0);
            if constexpr (SHAPE == SHORT) {
                if (there && !whole) {
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        if (e < it.count[v]) {
                            if constexpr (T == DT_F32) reinterpret_cast<uint32_t*>(base + head)[it.at[v] + e] = raw[v][e];
                            else reinterpret_cast<uint16_t*>(base + head)[it.at[v] + e] = (uint16_t)(raw[v][e >> 1] >> ((e & 1) * 16));
                        }
                }
            }
        }
    }
    __device__ __forceinline__ Pairs<VE> pairs(bool halves) const {
        Pairs<VE> x;
        each_pair<VE>(halves, [&](int e, int v0, int e0, int v1, int e1) {
            x.a[e] = Elem<T>::get(raw[v0], e0);
            x.b[e] = Elem<T>::get(raw[v1], e1);
        });
        return x;
    }
    __device__ __forceinline__ void round(bool halves, const Pairs<VE>& x) {
        if (halves) {
            raw[0] = Elem<T>::pack(x.a);
            raw[1] = Elem<T>::pack(x.b);
        } else {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float f[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) f[e] = e % 2 ? x.b[(v * VE + e) / 2] : x.a[(v * VE + e) / 2];
                raw[v] = Elem<T>::pack(f);
            }
        }
    }
    // An item's weights: T's or fp32, ones where there are none.
    static __device__ __forceinline__ Pairs<VE> weights(const char* w, int w_type, bool halves, const Item& it) {
        Pairs<VE> f;
#pragma unroll
        for (int e = 0; e < VE; ++e) f.a[e] = f.b[e] = 1.0f;
        if (w && w_type == T) {
            Vec<T, SHAPE> v;
            v.load(w, 0, true, it);
            f = v.pairs(halves);
        } else if (w) {
            const __amdgpu_buffer_rsrc_t rs = reach(w);
            each_pair<VE>(halves, [&](int e, int v0, int e0, int v1, int e1) {
                const uint32_t a = e0 < it.count[v0] ? 4 * (it.at[v0] + e0) : kNowhere, b = e1 < it.count[v1] ? 4 * (it.at[v1] + e1) : kNowhere;
                f.a[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, a, 0, 0));
                f.b[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, b, 0, 0));
            });
        }
        return f;
    }
};

// The angles of an item's pairs.
template <int VE, int SHAPE>
struct Angles {
    float c[VE], s[VE];
    __device__ __forceinline__ void load(const HeadsParams& p, int64_t pos, const Item& it) {
        const bool inside = pos >= 0 && pos < p.table;
        const int64_t row = inside ? pos * p.ldt * 4 : 0;
        const char *cos = reinterpret_cast<const char*>(p.cos) + row, *sin = reinterpret_cast<const char*>(p.sin) + row;
        const int pairs = p.neighbours ? 2 : 1;   // vectors that hold pairs of their own, of VE / pairs
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // the first and the second half of c and s
            constexpr int N = VE / 2;
            const int v = p.neighbours ? h : 0, from = it.at[v] / pairs + (p.neighbours ? 0 : h * N), count = it.count[v] / pairs - (p.neighbours ? 0 : h * N);
            take<N>(reach(cos, inside), reach(sin, inside), it.turns, from, count, h * N);
        }
        const float off = inside ? 0.0f : __builtin_nanf("");
#pragma unroll
        for (int e = 0; e < VE; ++e) c[e] += off, s[e] += off;
    }
    // N pairs from column `from` on, of which there are `count` (a short part's come one by one).
    template <int N>
    __device__ __forceinline__ void take(__amdgpu_buffer_rsrc_t cos, __amdgpu_buffer_rsrc_t sin, bool turns, int from, int count, int to) {
        if constexpr (SHAPE != SHORT) {
            const uint32_t at = turns && count > 0 ? 4 * from : kNowhere;
            if constexpr (N == 4) {
                const f32x4 a = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(cos, at, 0, 0));
                const f32x4 b = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(sin, at, 0, 0));
#pragma unroll
                for (int e = 0; e < 4; ++e) c[to + e] = a[e], s[to + e] = b[e];
            } else {
                const f32x2 a = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(cos, at, 0, 0));
                const f32x2 b = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(sin, at, 0, 0));
#pragma unroll
                for (int e = 0; e < 2; ++e) c[to + e] = a[e], s[to + e] = b[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint32_t at = turns && e < count ? 4 * (from + e) : kNowhere;
                c[to + e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(cos, at, 0, 0));
                s[to + e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sin, at, 0, 0));
            }
        }
    }
};
// Sum over the LPH lanes of a head, in each of them: neighbours within four lanes, eight and sixteen by data-parallel moves (where the
// lanes of a half already have the same sum, a mirror is as good as an exchange), further ones through LDS's crossbar.
template <int CTRL>
__device__ __forceinline__ float from_lane(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
    v += from_lane<0xB1>(v);                       // quad_perm [1, 0, 3, 2]
    v += from_lane<0x4E>(v);                       // quad_perm [2, 3, 0, 1]
    if constexpr (LPH >= 8) v += from_lane<0x141>(v);    // row_half_mirror
    if constexpr (LPH >= 16) v += from_lane<0x140>(v);   // row_mirror
    if constexpr (LPH >= 32) v += __shfl_xor(v, 16, 64);
    if constexpr (LPH >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}
// Products of an item's elements, those that it owns, added up (elements that there are not are zeros).
template <int VE, int SHAPE>
__device__ __forceinline__ float owned(bool halves, const Item& it, const Pairs<VE>& x, const Pairs<VE>& y) {
    float s = 0.0f;
    if constexpr (SHAPE == WHOLE) {
#pragma unroll
        for (int e = 0; e < VE; ++e) s = __builtin_fmaf(x.b[e], y.b[e], __builtin_fmaf(x.a[e], y.a[e], s));
    } else {
        each_pair<VE>(halves, [&](int e, int v0, int e0, int v1, int e1) {
            s += e0 >= it.first[v0] ? x.a[e] * y.a[e] : 0.0f;
            s += e1 >= it.first[v1] ? x.b[e] * y.b[e] : 0.0f;
        });
    }
    return s;
}

// 1 / sqrt(mean(x^2) + eps) of a head.  Where the sum of squares leaves fp32's range though the head does not, by the squares
// of x * 2^-80 or x * 2^80, as the norm of rows does it.
template <int VE, int SHAPE, int LPH, int IPL>
__device__ __forceinline__ float head_rstd(bool halves, const Item (&it)[IPL], const Pairs<VE> (&x)[IPL], float inv_dim, float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < IPL; ++i) sum += owned<VE, SHAPE>(halves, it[i], x[i], x[i]);
    sum = head_sum<LPH>(sum);
    const float mean = __builtin_fmaf(sum, inv_dim, eps);
    if (__builtin_expect(__builtin_isinf(sum) || mean < 0x1p-90f, 0)) {   // the same in every lane of the head
        const float by = __builtin_isinf(sum) ? 0x1p-80f : 0x1p80f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            Pairs<VE> scaled;
#pragma unroll
            for (int e = 0; e < VE; ++e) scaled.a[e] = x[i].a[e] * by, scaled.b[e] = x[i].b[e] * by;
            s += owned<VE, SHAPE>(halves, it[i], scaled, scaled);
        }
        return by / __builtin_sqrtf(head_sum<LPH>(s) * inv_dim + eps * by * by);
    }
    return __builtin_amdgcn_rsqf(mean);
}

// A step: 64 / LPH heads of a token, queries or keys.  A job: `per` steps of a token.  Waves take every so many-th job, so that at
// any time they are at neighbouring tokens (runs of tokens a wave measured 81 us instead of 71 on 16384 x (32 + 8) x 128 bf16).
struct Jobs {            // of a kind
    int steps, per, of;  // steps of a token, of a job; jobs of a token
    int wide;            // stride / of
    int64_t count;
    int narrow;          // stride % of
    int64_t stride;      // jobs between a wave's
};
struct BothJobs {
    Jobs of[2];
};
template <int LPH>
BothJobs jobs_of(const HeadsParams& p, int64_t waves) {   // waves: what the kinds have between them
    BothJobs b = {};
    for (int k = 0; k < 2; ++k) b.of[k].steps = (p.heads[k] + 64 / LPH - 1) / (64 / LPH);
    for (Jobs& j : b.of) {
        // whole tokens, whose angles are loaded once, but for jobs so few that waves would wait for the longest
        j.per = (int)std::max<int64_t>(1, std::min<int64_t>(j.steps, p.tokens * (b.of[0].steps + b.of[1].steps) / waves / kEach));
        j.of = (j.steps + j.per - 1) / j.per;
        j.count = p.tokens * j.of;
    }
    return b;
}
void set_stride(Jobs& j, int64_t stride) {
    j.stride = stride;
    j.wide = j.of ? (int)(stride / j.of) : 0;
    j.narrow = j.of ? (int)(stride % j.of) : 0;
}
// A position, read by the scalar unit (nothing here writes positions): a vector load's wait would be for the stores before it too.
__device__ __forceinline__ int64_t position(const int64_t* pos, int64_t token) {
    typedef const __attribute__((address_space(4))) int64_t* constant;
    return *(constant)(uintptr_t)(pos + token);
}
// A wave's way through the jobs of a kind.
struct Walk {
    Jobs jobs;
    int64_t j, token;    // job, and its token
    int part, step, to;  // the job's place among the token's, its step, its end
    __device__ __forceinline__ Walk(const Jobs& jobs_, int64_t first) : jobs(jobs_), j(first), token(0), part(0), step(0), to(0) {
        if (!there()) return;
        token = jobs.of == 1 ? j : j / jobs.of;
        part = (int)(j - token * jobs.of);
        begin();
    }
    __device__ __forceinline__ void begin() {
        step = part * jobs.per;
        to = min(step + jobs.per, jobs.steps);
    }
    __device__ __forceinline__ bool there() const { return j < jobs.count; }
    __device__ __forceinline__ bool more() const { return step + 1 < to; }   // steps of this job
    __device__ __forceinline__ void advance() {
        if (++step < to) return;
        j += jobs.stride;
        token += jobs.wide;
        part += jobs.narrow;
        if (part >= jobs.of) {
            part -= jobs.of;
            ++token;
        }
        begin();
    }
};
// The first of a step's heads.
template <int SZ, int G>
__device__ __forceinline__ char* first_head(const HeadsTensor& t, const Walk& w) {
    return const_cast<char*>(t.p) + (w.token * t.ld + (int64_t)w.step * G * t.hs) * SZ;
}

// The next step's heads are on their way while a wave has one's.
template <int T, int SHAPE, int LPH, int IPL>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(IPL == 1 ? 4 : 1)))
void heads_kernel(const HeadsParams p, const BothJobs jobs, float inv_dim) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE, G = 64 / LPH;
    const int lane = lane_id(), group = lane / LPH;
    const bool halves = !p.neighbours;
    Item it[IPL];
#pragma unroll
    for (int i = 0; i < IPL; ++i) it[i] = item_of<VE>(p, lane % LPH + LPH * i);
    int64_t first = (int64_t)blockIdx.x * kWaves + wave_id();   // (the keys' jobs follow the queries')
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        Walk at(jobs.of[k], first);
        if (!at.there()) {
            first -= at.jobs.count;
            continue;
        }
        const HeadsTensor xt = p.x[k], yt = p.y[k];
        const int heads = p.heads[k];
        const uint32_t x_off = (uint32_t)(group * (int)(xt.hs * SZ)), y_off = (uint32_t)(group * (int)(yt.hs * SZ));
        Vec<T, SHAPE> next[IPL];
        auto load = [&](const Walk& w) {
            const char* base = first_head<SZ, G>(xt, w);
            const bool there = w.there() && w.step * G + group < heads;
#pragma unroll
            for (int i = 0; i < IPL; ++i) next[i].load(base, x_off, there, it[i]);
        };
        load(at);
        Pairs<VE> w[IPL];
#pragma unroll
        for (int i = 0; i < IPL; ++i) w[i] = Vec<T, SHAPE>::weights(p.w[k], p.w_type, halves, it[i]);
        while (at.there()) {
            // a pair's factors: a' = a ca - b sb and b' = b cb + a sa; where nothing turns, ca and cb are the weights
            float ca[IPL][VE], sb[IPL][VE], cb[IPL][VE], sa[IPL][VE];
            const int64_t pos = p.rot ? position(p.pos, at.token) : 0;
#pragma unroll
            for (int i = 0; i < IPL; ++i) {
                Angles<VE, SHAPE> t;
                t.load(p, pos, it[i]);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    ca[i][e] = it[i].turns ? w[i].a[e] * t.c[e] : w[i].a[e];
                    cb[i][e] = it[i].turns ? w[i].b[e] * t.c[e] : w[i].b[e];
                    sa[i][e] = w[i].a[e] * t.s[e];
                    sb[i][e] = w[i].b[e] * t.s[e];
                }
            }
            bool more = true;
            while (more) {
                Pairs<VE> x[IPL];
#pragma unroll
                for (int i = 0; i < IPL; ++i) x[i] = next[i].pairs(halves);
                char* out = first_head<SZ, G>(yt, at);
                const bool mine = at.step * G + group < heads;
                more = at.more();
                at.advance();
                load(at);
                const float rstd = head_rstd<VE, SHAPE, LPH, IPL>(halves, it, x, inv_dim, p.eps);
#pragma unroll
                for (int i = 0; i < IPL; ++i) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float a = x[i].a[e] * rstd, b = x[i].b[e] * rstd;
                        x[i].a[e] = a * ca[i][e];
                        x[i].b[e] = b * cb[i][e];
                        if (it[i].turns) {
                            x[i].a[e] -= b * sb[i][e];
                            x[i].b[e] += a * sa[i][e];
                        }
                    }
                    Vec<T, SHAPE> y;
                    y.round(halves, x[i]);
                    y.store(out, y_off, mine, it[i]);
                }
            }
        }
        first = at.j - at.jobs.count;
    }
}

// dw of one kind stays in a lane's registers over all of its tokens: workgroups [0, q_parts) take the queries, the others the
// keys (where there is one workgroup, it takes both in turn).
template <int T, int SHAPE, int LPH, int IPL>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(IPL == 1 ? 3 : 1)))
void heads_bwd_kernel(const HeadsParams p, const BothJobs jobs, int q_parts, float inv_dim) {
    constexpr int VE = Elem<T>::VE, SZ = Elem<T>::SIZE, G = 64 / LPH;
    __shared__ float sums[kWaves * G * 2 * VE * LPH * IPL];   // of each wave and group, an element each
    const int lane = lane_id(), group = lane / LPH;
    const bool halves = !p.neighbours;
    Item it[IPL];
#pragma unroll
    for (int i = 0; i < IPL; ++i) it[i] = item_of<VE>(p, lane % LPH + LPH * i);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (p.parts > 1 && k != ((int)blockIdx.x >= q_parts)) continue;
        const HeadsTensor xt = p.x[k], dt = p.dy[k], yt = p.y[k];
        const int heads = p.heads[k];
        const uint32_t x_off = (uint32_t)(group * (int)(xt.hs * SZ)), d_off = (uint32_t)(group * (int)(dt.hs * SZ)),
                       y_off = (uint32_t)(group * (int)(yt.hs * SZ));
        Walk at(jobs.of[k], ((int64_t)blockIdx.x - (k && p.parts > 1 ? q_parts : 0)) * kWaves + wave_id());
        Vec<T, SHAPE> nx[IPL], nd[IPL];
        auto load = [&](const Walk& w) {
            const char *xb = first_head<SZ, G>(xt, w), *db = first_head<SZ, G>(dt, w);
            const bool there = w.there() && w.step * G + group < heads;
#pragma unroll
            for (int i = 0; i < IPL; ++i) nx[i].load(xb, x_off, there, it[i]);
#pragma unroll
            for (int i = 0; i < IPL; ++i) nd[i].load(db, d_off, there, it[i]);
        };
        load(at);
        Pairs<VE> w[IPL], dw[IPL];
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            w[i] = Vec<T, SHAPE>::weights(p.w[k], p.w_type, halves, it[i]);
#pragma unroll
            for (int e = 0; e < VE; ++e) dw[i].a[e] = dw[i].b[e] = 0.0f;
        }
        while (at.there()) {
            const int64_t pos = p.rot ? position(p.pos, at.token) : 0;
            Angles<VE, SHAPE> turn[IPL];
#pragma unroll
            for (int i = 0; i < IPL; ++i) turn[i].load(p, pos, it[i]);
            bool more = true;
            while (more) {
                Pairs<VE> x[IPL], g[IPL];
#pragma unroll
                for (int i = 0; i < IPL; ++i) {
                    x[i] = nx[i].pairs(halves);
                    g[i] = nd[i].pairs(halves);
                }
                char* out = first_head<SZ, G>(yt, at);
                const bool mine = at.step * G + group < heads;
                more = at.more();
                at.advance();
                load(at);
                const float rstd = head_rstd<VE, SHAPE, LPH, IPL>(halves, it, x, inv_dim, p.eps);
                float through = 0.0f;
#pragma unroll
                for (int i = 0; i < IPL; ++i) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float a = g[i].a[e], b = g[i].b[e];
                        if (it[i].turns) {
                            g[i].a[e] = a * turn[i].c[e] + b * turn[i].s[e];
                            g[i].b[e] = b * turn[i].c[e] - a * turn[i].s[e];
                        }
                        x[i].a[e] *= rstd;
                        x[i].b[e] *= rstd;
                        if (mine) {
                            dw[i].a[e] = __builtin_fmaf(g[i].a[e], x[i].a[e], dw[i].a[e]);
                            dw[i].b[e] = __builtin_fmaf(g[i].b[e], x[i].b[e], dw[i].b[e]);
                        }
                        g[i].a[e] *= w[i].a[e];
                        g[i].b[e] *= w[i].b[e];
                    }
                    through += owned<VE, SHAPE>(halves, it[i], g[i], x[i]);
                }
                through = head_sum<LPH>(through) * inv_dim * rstd;
#pragma unroll
                for (int i = 0; i < IPL; ++i) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        g[i].a[e] = __builtin_fmaf(-x[i].a[e], through, g[i].a[e] * rstd);
                        g[i].b[e] = __builtin_fmaf(-x[i].b[e], through, g[i].b[e] * rstd);
                    }
                    Vec<T, SHAPE> y;
                    y.round(halves, g[i]);
                    y.store(out, y_off, mine, it[i]);
                }
            }
        }
        if (!p.dw[k]) continue;   // the same in every thread
        // (lanes whose vectors overlap have the same sums there, and store the same)
        float* own = sums + (wave_id() * G + group) * p.dim;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            each_pair<VE>(halves, [&](int e, int v0, int e0, int v1, int e1) {
                if (e0 < it[i].count[v0]) own[it[i].at[v0] + e0] = dw[i].a[e];
                if (e1 < it[i].count[v1]) own[it[i].at[v1] + e1] = dw[i].b[e];
            });
        __syncthreads();
        float* to = p.parts > 1 ? p.part + (int64_t)blockIdx.x * p.dim : p.dw[k];
        for (int e = threadIdx.x; e < p.dim; e += 64 * kWaves) {
            float s = 0.0f;
#pragma unroll 8
            for (int q = 0; q < kWaves * G; ++q) s += sums[q * p.dim + e];
            to[e] = s;
        }
        __syncthreads();
    }
}

// dw = the parts' sums in order: 64 elements of queries' or keys' weights a workgroup, every sixteenth part a wave.
__global__ __launch_bounds__(1024) void heads_join_kernel(const HeadsParams p, int q_parts) {
    __shared__ float sums[16][64];
    const int k = blockIdx.y, e = (int)blockIdx.x * 64 + lane_id(), w = wave_id();
    if (!p.dw[k]) return;
    const int first = k ? q_parts : 0, end = k ? p.parts : q_parts;
    float s = 0.0f;
    if (e < p.dim) {
#pragma unroll 8
        for (int i = first + w; i < end; i += 16) s += p.part[(int64_t)i * p.dim + e];
    }
    sums[w][lane_id()] = s;
    __syncthreads();
    if (w != 0 || e >= p.dim) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sums[i][lane_id()];
    p.dw[k][e] = s;
}

template <int VE>
int shape_of(const HeadsParams& p) {
    const int parts[2] = {p.neighbours ? p.rot : p.rot / 2, p.dim - p.rot};
    int shape = WHOLE;
    for (int n : parts)
        if (n % VE) shape = std::max<int>(shape, n < VE ? SHORT : OVERLAP);
    return shape;
}
int items_in(int type, const HeadsParams& p) {
    return type == DT_F32 ? items_of<4>(p.dim, p.rot, p.neighbours) : items_of<8>(p.dim, p.rot, p.neighbours);
}
// Lanes of a head.  A wave that takes several heads holds their offsets from the first in 32 bits: heads further apart go one to a
// wave.
int lanes_of(int type, const HeadsParams& p) {
    for (int k = 0; k < 2; ++k)
        for (const HeadsTensor* h : {&p.x[k], &p.dy[k], &p.y[k]})
            if (h->hs >= int64_t(1) << 24) return 64;
    const int items = items_in(type, p);
    int lanes = 4;
    while (lanes < items && lanes < 64) lanes *= 2;
    return lanes;
}
// f(type, shape, lanes of a head, items of a lane); a head of 1024 has 128 items of fp32 and up to two more where its parts
// end inside a vector.
template <class F>
hipError_t by_size(int type, const HeadsParams& p, F&& f) {
    auto sized = [&](auto t, auto s) {
        typedef std::integral_constant<int, 1> One;
        switch (lanes_of(type, p)) {
            case 4: return f(t, s, std::integral_constant<int, 4>{}, One{});
            case 8: return f(t, s, std::integral_constant<int, 8>{}, One{});
            case 16: return f(t, s, std::integral_constant<int, 16>{}, One{});
            case 32: return f(t, s, std::integral_constant<int, 32>{}, One{});
        }
        if (items_in(type, p) <= 64) return f(t, s, std::integral_constant<int, 64>{}, One{});
        return f(t, s, std::integral_constant<int, 64>{}, std::integral_constant<int, 3>{});
    };
    auto shaped = [&](auto t) {
        switch (type == DT_F32 ? shape_of<4>(p) : shape_of<8>(p)) {
            case WHOLE: return sized(t, std::integral_constant<int, WHOLE>{});
            case OVERLAP: return sized(t, std::integral_constant<int, OVERLAP>{});
            default: return sized(t, std::integral_constant<int, SHORT>{});
        }
    };
    if (type == DT_F32) return shaped(std::integral_constant<int, DT_F32>{});
    if (type == DT_BF16) return shaped(std::integral_constant<int, DT_BF16>{});
    return shaped(std::integral_constant<int, DT_F16>{});
}
int steps_of(int lanes, int heads) { return (heads + 64 / lanes - 1) / (64 / lanes); }

}  // namespace

// As many workgroups as the card holds at once, so that what a wave sets up it does once.
hipError_t launch_heads(int in_type, const HeadsParams& p, hipStream_t st) {
    return by_size(in_type, p, [&](auto t, auto s, auto l, auto n) {
        const int64_t most = 4 * (int64_t)num_compute_units();
        BothJobs jobs = jobs_of<decltype(l)::value>(p, most * kWaves);
        const int64_t grid = std::min<int64_t>((jobs.of[0].count + jobs.of[1].count + kWaves - 1) / kWaves, most);
        for (Jobs& j : jobs.of) set_stride(j, grid * kWaves);
        hipLaunchKernelGGL((heads_kernel<decltype(t)::value, decltype(s)::value, decltype(l)::value, decltype(n)::value>),
                           dim3((unsigned)grid), dim3(64 * kWaves), 0, st, p, jobs, 1.0f / (float)p.dim);
        return hipGetLastError();
    });
}

int heads_bwd_most_parts(const HeadsParams& p) {   // for any rotation and strides: a head a wave
    return (int)std::max<int64_t>(1, std::min<int64_t>((p.tokens * (p.heads[0] + p.heads[1]) + kWaves - 1) / kWaves, 3 * (int64_t)num_compute_units()));
}
// A step a wave, or as many waves as the card holds at once.
int heads_bwd_parts(int in_type, const HeadsParams& p) {
    const int lanes = lanes_of(in_type, p);
    const int64_t steps = p.tokens * (steps_of(lanes, p.heads[0]) + steps_of(lanes, p.heads[1]));
    return (int)std::max<int64_t>(1, std::min<int64_t>((steps + kWaves - 1) / kWaves, 3 * (int64_t)num_compute_units()));
}

hipError_t launch_heads_bwd(int in_type, const HeadsParams& p, hipStream_t st) {
    // parts of the queries and of the keys by their steps, one of each at least where there are some
    const int lanes = lanes_of(in_type, p);
    const int64_t of_q = steps_of(lanes, p.heads[0]), of_k = steps_of(lanes, p.heads[1]);
    int q_parts = (int)(p.parts * of_q / std::max<int64_t>(1, of_q + of_k));
    if (p.heads[0] > 0) q_parts = std::max(q_parts, 1);
    if (p.heads[1] > 0) q_parts = std::min(q_parts, p.parts - 1);
    const hipError_t e = by_size(in_type, p, [&](auto t, auto s, auto l, auto n) {
        BothJobs jobs = jobs_of<decltype(l)::value>(p, (int64_t)p.parts * kWaves);
        for (int k = 0; k < 2; ++k) set_stride(jobs.of[k], (int64_t)kWaves * (p.parts == 1 ? 1 : k ? p.parts - q_parts : q_parts));
        hipLaunchKernelGGL((heads_bwd_kernel<decltype(t)::value, decltype(s)::value, decltype(l)::value, decltype(n)::value>),
                           dim3((unsigned)p.parts), dim3(64 * kWaves), 0, st, p, jobs, q_parts, 1.0f / (float)p.dim);
        return hipGetLastError();
    });
    if (e != hipSuccess || p.parts == 1 || (!p.dw[0] && !p.dw[1])) return e;
    hipLaunchKernelGGL(heads_join_kernel, dim3((unsigned)((p.dim + 63) / 64), 2), dim3(1024), 0, st, p, q_parts);
    return hipGetLastError();
}

}  // namespace gemm
