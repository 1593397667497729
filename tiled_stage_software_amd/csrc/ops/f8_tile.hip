// f8_tile.hip -- the 8-bit product on tiles: BM x BN of C per workgroup, slabs of 128
// bytes of K in a two-slot LDS ring, v_mfma_f32_16x16x128_f8f6f4 (or its bf16 form for fp32
// results) on 16 x 16 blocks.
//
// A 128-byte slab of e4m3 and a 64-element slab of bf16 are the same bytes per LDS row, per copy
// and per matrix-core cycle, so the ring, its loaders and the epilogues are those of the 16-bit
// kernels.  What differs is the fragment: 32 bytes a lane, a whole slab of K in one instruction.
// Holding a slab's fragments twice (as the 16-bit kernels hold a k-step's) would take 192
// registers beside the 128 accumulators; so a slab is cut along M instead of K: step s multiplies AH
// blocks of A's rows with all of the wave's B, only A's fragments are doubled, and B's are
// read anew for the next slab in the last step, each right after its last use.
#include <algorithm>

#include "f8_common.hpp"
#include "short_loader.hpp"

namespace gemm {
namespace {

constexpr int kSlabBytes = 128;

template <int BM, int BN, int WM, int WN, int KS, bool WIDE>
struct F8Compute : MfmaCompute<__bf16, BM, BN, 64, WM, WN, 16> {
    typedef MfmaCompute<__bf16, BM, BN, 64, WM, WN, 16> C;
    static constexpr int AH = C::TM / KS;   // blocks of A's rows in a step
    static_assert(C::ROWB == kSlabBytes && C::TM % KS == 0, "whole blocks in a step");
    i32x8 ra[2][AH], rb[C::TN];
    uint32_t oa[2], ob[2];                  // LDS offsets of a lane's two chunks (row 0 of the wave's tile)
    LDS_AS const char* next_a;              // what frag() asked for; the next math() reads it
    LDS_AS const char* next_b;
    bool ask_a = false, ask_b = false;

    __device__ __forceinline__ void init(LDS_AS char* smem_) {
        this->smem = smem_;
        const int w = wave_id(), lane = lane_id();
        const int r = lane % 16, g = lane / 16, kc = (g & 1) * 2 + (g >> 1);   // chunk order: no bank conflicts
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = (uint32_t)(r * kSlabBytes + (((kc + 4 * h) ^ swz<8>(r)) << 4));
            oa[h] = (uint32_t)(w / WN * C::WTM * kSlabBytes) + at;
            ob[h] = (uint32_t)(C::A_BYTES + w % WN * C::WTN * kSlabBytes) + at;
        }
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int j = 0; j < C::TN; ++j) this->acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    static __device__ __forceinline__ i32x8 read(LDS_AS const char* st, const uint32_t* o, int block) {
        return join16(*reinterpret_cast<LDS_AS const u32x4*>(st + o[0] + block * 16 * kSlabBytes),
                      *reinterpret_cast<LDS_AS const u32x4*>(st + o[1] + block * 16 * kSlabBytes));
    }
    // Step ks of a slab: its blocks of A, at step 0 with the slab's B.  Read at once for slab 0 (nothing
    // is multiplied yet), else by the math() that follows.
    template <int BUF>
    __device__ __forceinline__ void frag(int slab, int slot, int ks) {
        LDS_AS const char* st = this->smem + slot * C::STAGE;
        next_a = st + ks * AH * 16 * kSlabBytes;
        next_b = st;
        if (slab == 0 && ks == 0) {
#pragma unroll
            for (int i = 0; i < AH; ++i) ra[BUF][i] = read(next_a, oa, i);
#pragma unroll
            for (int j = 0; j < C::TN; ++j) rb[j] = read(st, ob, j);
        } else {
            ask_a = true;
            ask_b = ks == 0;
        }
    }
    // Column by column of the wave's B: the products of this step, then the reads.  A's come with the
    // first columns, so that the last of them has the rest of the step to arrive.
    template <int BUF, class Between>
    __device__ __forceinline__ void step(int ks, Between&& between) {
        constexpr int PER = (2 * AH + C::TN - 1) / C::TN > 1 ? 2 : 1;   // A blocks read with a column
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
#pragma unroll
            for (int i = 0; i < AH; ++i)
                this->acc[ks * AH + i][j] = mfma_f8<WIDE>(rb[j], ra[BUF][i], this->acc[ks * AH + i][j]);
            if (ask_a) {
#pragma unroll
                for (int i = 0; i < AH; ++i)
                    if (i / PER == j) ra[BUF ^ 1][i] = read(next_a, oa, i);
            }
            if (ask_b) rb[j] = read(next_b, ob, j);
            between(j);
            __builtin_amdgcn_sched_barrier(0);
        }
        ask_a = ask_b = false;
    }
    __device__ __forceinline__ void wait_lds() { wait_lgkm0(); }
    __device__ __forceinline__ void barrier() { gemm::barrier(); }

    // The accumulators times their scales (rows past M and columns past N are not stored).
    __device__ __forceinline__ void scale(const float* sa, const float* sb, const GemmParams& p, int m0, int n0) {
        const int w = wave_id(), lane = lane_id();
        const int m = m0 + w / WN * C::WTM + lane % 16, n = n0 + w % WN * C::WTN + 4 * (lane / 16);
        float fb[C::TN][4];
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) fb[j][e] = scale_or_one(sb, min(n + 16 * j + e, p.N - 1));
#pragma unroll
        for (int i = 0; i < C::TM; ++i) {
            const float f = scale_or_one(sa, min(m + 16 * i, p.M - 1));
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) this->acc[i][j][e] = this->acc[i][j][e] * f * fb[j][e];
        }
    }
};

// Direct global -> LDS copies by the first NC waves: 16-byte aligned rows, whole slabs and tiles.
template <int S, int BM, int BN, int WM, int WN, int KS, bool WIDE, int NC, bool COPY>
struct F8RingOps : F8Compute<BM, BN, WM, WN, KS, WIDE> {
    typedef F8Compute<BM, BN, WM, WN, KS, WIDE> F;
    ALoader<BM, kSlabBytes, NC> la;
    DirectLoader<BN, kSlabBytes, NC, true> lb;
    static constexpr int LA = decltype(la)::IPW, L = LA + decltype(lb)::IPW;
    int slab_ = 0, slot_ = 0;
    bool ask_copy = false;
    __device__ __forceinline__ void copies(int slab, int slot, int c0, int c1) {
        LDS_AS char* st = this->smem + slot * F::C::STAGE;
        la.issue(slab, st, c0, c1 < LA ? c1 : LA);
        lb.issue(slab, st + F::C::A_BYTES, c0 > LA ? c0 - LA : 0, c1 - LA);
    }
    // the prologue's slabs go out at once, the others between the next math()'s products
    __device__ __forceinline__ void issue(int slab, int slot, int, int) {
        if (!COPY) return;
        if (slab < S) { copies(slab, slot, 0, L); return; }
        slab_ = slab; slot_ = slot; ask_copy = true;
    }
    template <int N>
    __device__ __forceinline__ void wait_slabs() { if (COPY) wait_vm<N * L>(); }
    template <int BUF, int HAS, int PARTS>
    __device__ __forceinline__ void math(int ks) {
        constexpr int TN = F::C::TN;
        this->template step<BUF>(ks, [&](int j) {
            if (COPY && HAS && ask_copy) copies(slab_, slot_, j * L / TN, (j + 1) * L / TN);
        });
        ask_copy = false;
    }
};

// Any pitch, alignment and K >= 128: 16-byte loads of any alignment into registers, AHEAD slabs ahead,
// written into the other slot in the last step but one.  A last slab that K does not fill is
// the row's last 128 bytes, with zeros in A for what earlier slabs had.  Rows past the end
// repeat the last (CLAMP), or there are none: the tile lies inside both operands.
template <int BM, int BN, int WM, int WN, int KS, bool WIDE, bool CLAMP>
struct F8StagedOps : F8Compute<BM, BN, WM, WN, KS, WIDE> {
    typedef F8Compute<BM, BN, WM, WN, KS, WIDE> F;
    static constexpr int NT = 64 * WM * WN, STEP = NT / 8;
    static constexpr int CA = BM / STEP, CH = (BM + BN) / STEP;   // chunks per thread and slab
    static_assert(BM % STEP == 0 && BN % STEP == 0 && STEP % 16 == 0, "rows split evenly; one swizzle phase per thread");
    static_assert(KS >= 4, "the write is not in the step of the load");
    const uint8_t* base[2];
    int64_t ld[2];
    uint32_t off[CLAMP ? CH : 2];
    uint32_t dst;
    static constexpr int AHEAD = BM < 256 && !(WIDE && NT == 256) ? 2 : 1;   // slabs in registers (where two fit)
    u32x4 v[AHEAD][CH], mask = {~0u, ~0u, ~0u, ~0u};
    int K;              // bytes of this workgroup's part of the rows
    __device__ __forceinline__ void init_rows(const uint8_t* A, int64_t lda, int m0, int M, const uint8_t* B, int64_t ldb,
                                              int n0, int N) {
        const int row = (int)threadIdx.x / 8, c = (int)threadIdx.x % 8;
        base[0] = A + (int64_t)m0 * lda;
        base[1] = B + (int64_t)n0 * ldb;
        ld[0] = lda;
        ld[1] = ldb;
        if constexpr (CLAMP) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                off[i] = (i < CA ? (uint32_t)min(row + i * STEP, M - 1 - m0) * (uint32_t)lda
                                 : (uint32_t)min(row + (i - CA) * STEP, N - 1 - n0) * (uint32_t)ldb) + 16 * c;
        } else {
            off[0] = (uint32_t)row * (uint32_t)lda + 16 * c;
            off[1] = (uint32_t)row * (uint32_t)ldb + 16 * c;
        }
        dst = (uint32_t)(row * kSlabBytes + ((c ^ swz<8>(row)) << 4));
    }
    template <int V>
    __device__ __forceinline__ void load(int slab) {
        int k = slab * kSlabBytes;
        if (k + kSlabBytes > K) {
            const int old = k + kSlabBytes - K - (int)threadIdx.x % 8 * 16;   // bytes of this chunk that earlier slabs had
            k = K - kSlabBytes;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int o = old - 4 * q;
                mask[q] = o >= 4 ? 0u : o <= 0 ? ~0u : ~0u << (8 * o);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if constexpr (CLAMP) v[V][i] = load16(base[i >= CA] + k + off[i]);
            else v[V][i] = load16(base[i >= CA] + (k + (i >= CA ? i - CA : i) * STEP * ld[i >= CA]) + off[i >= CA]);
        }
    }
    template <int V>
    __device__ __forceinline__ void put(int i, int slot, bool last) {   // (the mask is the last slab's; one slab ahead, whole until then)
        u32x4 x = v[V][i];
        if (i < CA && (AHEAD == 1 || last)) x &= mask;
        *reinterpret_cast<LDS_AS u32x4*>(this->smem + slot * F::C::STAGE + dst + i * STEP * kSlabBytes) = x;
    }
    // Multiplies slab kt out of its slot, kt mod 2.  Slab kt + AHEAD is loaded into registers V; slab kt + 1 goes from
    // registers W to the other slot, which the barrier before this slab freed.
    template <int V, int W, bool LAST>
    __device__ __forceinline__ void slab(int kt, int slabs) {
        const int slot = kt & 1;
        if (!LAST) load<V>(AHEAD == 1 ? kt + 1 : min(kt + 2, slabs - 1));
        const bool last = kt + 2 == slabs;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks < KS - 1) {
                if (ks % 2 == 0) this->template frag<1>(kt, slot, ks + 1);
                else this->template frag<0>(kt, slot, ks + 1);
            } else if (!LAST) {
                this->wait_lds();
                this->barrier();
                this->template frag<0>(kt + 1, slot ^ 1, 0);
            }
            auto between = [&](int j) {
                if (LAST || ks != KS - 2) return;
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (i * F::C::TN / CH == j) put<W>(i, slot ^ 1, last);
            };
            if (ks % 2 == 0) this->template step<0>(ks, between);
            else this->template step<1>(ks, between);
        }
    }
    __device__ __forceinline__ void run(int slabs) {
        load<0>(0);
        if constexpr (AHEAD == 2) load<1>(min(1, slabs - 1));
#pragma unroll
        for (int i = 0; i < CH; ++i) put<0>(i, 0, slabs == 1);
        this->wait_lds();
        this->barrier();
        this->template frag<0>(0, 0, 0);
        int kt = 0;
        if constexpr (AHEAD == 1) {
            for (; kt + 1 < slabs; ++kt) slab<0, 0, false>(kt, slabs);
            slab<0, 0, true>(kt, slabs);
        } else {
            for (; kt + 2 < slabs; kt += 2) {
                slab<0, 1, false>(kt, slabs);
                slab<1, 0, false>(kt + 1, slabs);
            }
            if (kt + 2 == slabs) {
                slab<0, 1, false>(kt, slabs);
                slab<1, 0, true>(kt + 1, slabs);
            } else {
                slab<0, 1, true>(kt, slabs);
            }
        }
    }
};

struct F8Extra {
    const float* sa;
    const float* sb;
    int per_split;     // slabs of K per split
    int64_t part;      // bytes between the splits' results
};

// OUT: type of what is stored; S: slots of the ring (0: staged loads).  Splits of K (blockIdx.y) store plain sums,
// each into its own buffer.
template <int OUT, int BM, int BN, int WM, int WN, int KS, bool WIDE, int S>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2)))
void f8_tile_kernel(GemmParams p, const F8Extra x) {
    constexpr int NW = WM * WN, NC = NW < 4 ? NW : 4;
    constexpr int RING = (S > 0 ? S : 2) * (BM + BN) * kSlabBytes, EPI = (OUT != DT_F32 && BN == 256) ? BM * BN * 2 : 0;
    __shared__ __attribute__((aligned(1024))) char smem_raw[RING > EPI ? RING : EPI];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m_keep = tm * BM, n_keep = tn * BN;
    const int m0 = max(0, min(m_keep, p.M - BM)), n0 = max(0, min(n_keep, p.N - BN));
    const int s0 = (int)blockIdx.y * x.per_split;
    const int K = min(p.K - s0 * kSlabBytes, x.per_split * kSlabBytes);
    const int slabs = (K + kSlabBytes - 1) / kSlabBytes;
    const uint8_t* A = reinterpret_cast<const uint8_t*>(p.A) + s0 * kSlabBytes;
    const uint8_t* B = reinterpret_cast<const uint8_t*>(p.B) + s0 * kSlabBytes;
    p.C += (int64_t)blockIdx.y * x.part;
    auto finish = [&](auto& ops) {
        if (x.sa || x.sb) ops.scale(x.sa, x.sb, p, m0, n0);
        if constexpr (EPI > 0) {
            if (p.beta == 0.0f && m0 == m_keep && n0 == n_keep && m0 + BM <= p.M && n0 + BN <= p.N &&
                (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 && (p.ldc * 2) % 16 == 0) {
                ops.template epilogue_lds<OUT, 64 * NW>(p, m0, n0);
                return;
            }
        }
        ops.template epilogue<OUT>(p, m0, n0, m_keep, n_keep);
    };
    if constexpr (S > 0) {
        if (NC == NW || wave_id() < NC) {
            F8RingOps<S, BM, BN, WM, WN, KS, WIDE, NC, true> ops;
            ops.init(smem);
            init_a<BM, kSlabBytes, NC>(ops.la, reinterpret_cast<const char*>(A) + (int64_t)m0 * p.lda, p.lda, kSlabBytes, p.M - m0);
            ops.lb.init(reinterpret_cast<const char*>(B) + (int64_t)n0 * p.ldb, p.ldb, kSlabBytes);
            gemm_sched::ring_mainloop<S, KS, 1>(ops, slabs);
            finish(ops);
        } else if constexpr (NC < NW) {
            F8RingOps<S, BM, BN, WM, WN, KS, WIDE, NC, false> ops;
            ops.init(smem);
            gemm_sched::ring_mainloop<S, KS, 1>(ops, slabs);
            finish(ops);
        }
    } else {
        F8StagedOps<BM, BN, WM, WN, KS, WIDE, (BM < 256)> ops;
        ops.init(smem);
        ops.init_rows(A, p.lda, m0, p.M, B, p.ldb, n0, p.N);
        ops.K = K;
        ops.run(slabs);
        finish(ops);
    }
}

// C = alpha * diag(sa) * (sum of the splits, in order) * diag(sb) + beta * C
template <int OUT>
__global__ __launch_bounds__(256) void f8_join_kernel(const GemmParams p, const F8Extra x, const char* part, int ldp, int splits) {
    const int64_t quads = ldp / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= quads * p.M) return;
    const int64_t m = id / quads;
    const int n = (int)(id % quads) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < splits; ++i)
        s += *reinterpret_cast<const f32x4*>(part + i * x.part + (m * ldp + n) * 4);
    const float a = scale_or_one(x.sa, m);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = s[e] * a * scale_or_one(x.sb, min(n + e, p.N - 1));
    store4<OUT>(p, m, n, s);
}

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct F8Plan {
    int bm, bn;    // rows and columns of a tile: 256 x 256, 128 x 128 or 64 x 128
    int splits;
};

// The tile with the least time on the fullest compute unit: a 256 x 256 tile costs four units and a 128 x 128 one
// kSmallCost (both measured on 4096 x 4096 x 4096 and 8192^3).  Where small tiles do not fill the card: the height
// and the splits of K that should be fastest.  A slab takes slab_us() on a compute unit that has nothing else to hide its
// loads with; more workgroups than units share them at kShared; a split writes and reads its fp32
// sums once (at the rate of a copy) and needs one more launch.
constexpr double kSmallCost = 1.35, kShared = 0.75, kJoinUs = 4.0, kBytesPerUs = 4.5e6;
double slab_us(int bm, bool wide) { return bm == 64 ? (wide ? 0.6 : 0.35) : (wide ? 1.05 : 0.5); }   // 112 to 256 workgroups, 16 to 32 slabs
double staged_us(int bm) { return bm == 256 ? 1.0 : bm == 128 ? 0.5 : 0.4; }   // longer from rows of any alignment
double rounds_of(int64_t workgroups) {
    const int64_t cu = num_compute_units();
    return workgroups <= cu ? 1.0 : kShared * ceil_div(workgroups, cu);
}
int64_t f8_ldp(int64_t N) { return (N + 3) / 4 * 4; }
F8Plan f8_plan(int64_t M, int64_t N, int64_t K, bool wide) {
    F8Plan q = {128, 128, 1};
    const int64_t cu = num_compute_units();
    const int64_t t256 = ceil_div(M, 256) * ceil_div(N, 256), t128 = ceil_div(M, 128) * ceil_div(N, 128);
    if (!wide && M >= 256 && N >= 256 && ceil_div(t256, cu) * 4.0 <= ceil_div(t128, cu) * kSmallCost) return F8Plan{256, 256, 1};
    if (t128 > cu && M > kShortRows) return q;
    const int64_t slabs = ceil_div(K, kSlabBytes);
    double best = 0.0;
    for (int bm = 128; bm >= 64; bm -= 64) {
        const int64_t tiles = ceil_div(M, bm) * ceil_div(N, 128);
        for (int64_t s = 1; s <= 16 && s * 4 <= slabs + 3; ++s) {
            const double us = rounds_of(tiles * s) * ceil_div(slabs, s) * slab_us(bm, wide) +
                              (s > 1 ? kJoinUs + s * (double)M * f8_ldp(N) * 8.0 / kBytesPerUs : 0.0);
            if (best == 0.0 || us < best) {
                best = us;
                q.bm = bm;
                q.splits = (int)s;
            }
        }
    }
    return q;
}

// Whether the launch that copies (`bytes` of copies) costs less than the staged loads' slower slabs.
bool f8_copy_pays(const F8Plan& q, const F8Params& f, int64_t slabs, size_t bytes) {
    const double rounds = rounds_of(ceil_div(f.M, q.bm) * ceil_div(f.N, q.bn) * q.splits);
    return kJoinUs + 2.0 * bytes / kBytesPerUs < rounds * ceil_div(slabs, q.splits) * staged_us(q.bm);
}

template <int OUT, int BM, int BN, int WM, int WN, bool WIDE, int S>
hipError_t go(const GemmParams& p, const F8Extra& x, int splits, hipStream_t st) {
    hipLaunchKernelGGL((f8_tile_kernel<OUT, BM, BN, WM, WN, 4, WIDE, S>), dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)splits),
                       dim3(64 * WM * WN), 0, st, p, x);
    return hipGetLastError();
}
// Small tiles that have a compute unit to themselves: eight waves, so that two on a SIMD take turns, and four slots, so that
// three slabs are on their way.  Else a second workgroup, which two slots leave room for, does both.
template <int OUT, bool WIDE>
hipError_t tile_of(const F8Plan& q, bool direct, const GemmParams& p, const F8Extra& x, hipStream_t st) {
    if constexpr (!WIDE) {
        if (q.bm == 256) return direct ? go<OUT, 256, 256, 2, 4, WIDE, 2>(p, x, q.splits, st) : go<OUT, 256, 256, 2, 4, WIDE, 0>(p, x, q.splits, st);
    }
    const bool alone = (int64_t)p.tiles_m * p.tiles_n * q.splits <= num_compute_units();
    if (q.bm == 64) {
        if (!direct) return go<OUT, 64, 128, 1, 8, WIDE, 0>(p, x, q.splits, st);
        return alone ? go<OUT, 64, 128, 1, 8, WIDE, 4>(p, x, q.splits, st) : go<OUT, 64, 128, 1, 8, WIDE, 2>(p, x, q.splits, st);
    }
    if (!direct) return alone ? go<OUT, 128, 128, 2, 4, WIDE, 0>(p, x, q.splits, st) : go<OUT, 128, 128, 2, 2, WIDE, 0>(p, x, q.splits, st);
    return alone ? go<OUT, 128, 128, 2, 4, WIDE, 4>(p, x, q.splits, st) : go<OUT, 128, 128, 2, 2, WIDE, 2>(p, x, q.splits, st);
}
template <int OUT>
hipError_t join_of(const GemmParams& p, const F8Extra& x, const void* part, int64_t ldp, int splits, hipStream_t st) {
    hipLaunchKernelGGL(f8_join_kernel<OUT>, dim3((unsigned)ceil_div(p.M * ldp / 4, 256)), dim3(256), 0, st, p, x,
                       static_cast<const char*>(part), (int)ldp, splits);
    return hipGetLastError();
}

}  // namespace

constexpr size_t kMostCopied = size_t(1) << 34;   // rows_pack counts chunks in 32 bits

// K >= 128 and strides that the tiles' 32-bit offsets hold (256 rows below 2^31 bytes).
bool f8_tile_fits(const F8Params& f) {
    const int64_t most = int64_t(1) << 22;
    return f.K >= kSlabBytes && f.lda <= most && f.ldb <= most && ceil_div(f.M, 128) * ceil_div(f.N, 128) < (int64_t(1) << 22);
}

namespace {

// What a call does with the workspace it has.
struct F8Launch {
    F8Plan q;
    int per_split;       // slabs of a split
    int64_t each, kp;    // bytes of a split's sums; K in whole slabs
    RowsJob ja, jb;      // copies of the operands, behind the splits' sums ...
    bool copy_a, copy_b; // ... of those that the direct copies cannot take
    size_t used, wants;
    bool copies, direct;
};
F8Launch f8_launch_of(const F8Params& f, size_t ws_bytes) {
    F8Launch l;
    F8Plan& q = l.q;
    q = f8_plan(f.M, f.N, f.K, f.out_type == DT_F32);
    const int64_t slabs = ceil_div(f.K, kSlabBytes);
    l.each = (int64_t)f.M * f8_ldp(f.N) * sizeof(float);
    if (q.splits > 1 && ws_bytes < (size_t)(q.splits * l.each)) q.splits = (int)(ws_bytes / l.each);
    if (q.splits < 2) q.splits = 1;
    l.per_split = (int)ceil_div(slabs, q.splits);
    q.splits = (int)ceil_div(slabs, l.per_split);
    l.kp = slabs * kSlabBytes;
    const int64_t least_a = least_rows(q.bm), least_b = q.bn;
    l.ja = {f.A, nullptr, f.lda, f.M, f.K, std::max((int64_t)f.M, least_a), l.kp};
    l.jb = {f.B, nullptr, f.ldb, f.N, f.K, std::max((int64_t)f.N, least_b), l.kp};
    l.copy_a = f.M < least_a || f.K != l.kp || ((uintptr_t)f.A | f.lda) % 16;
    l.copy_b = f.N < least_b || f.K != l.kp || ((uintptr_t)f.B | f.ldb) % 16;
    l.used = q.splits > 1 ? ((size_t)(q.splits * l.each) + 255) & ~size_t(255) : 0;
    l.wants = l.used + (l.copy_a ? l.ja.bytes() : 0) + (l.copy_b ? l.jb.bytes() : 0);
    l.copies = (l.copy_a || l.copy_b) && l.wants <= ws_bytes && l.wants < kMostCopied && f8_copy_pays(q, f, slabs, l.wants - l.used);
    l.direct = l.copies || (!l.copy_a && !l.copy_b);
    return l;
}

}  // namespace

// Bytes for the splits and for the copies of contiguous operands that the call would make.
size_t f8_tile_workspace(const F8Params& f) {
    const F8Launch l = f8_launch_of(f, SIZE_MAX / 2);
    return l.copies ? l.wants : l.used;
}

// Expected microseconds of few rows: rounds of slabs and the launches beside them, or reading B (5 TB/s).
double f8_tile_us(const F8Params& f, size_t ws_bytes) {
    const F8Launch l = f8_launch_of(f, ws_bytes);
    const double slab = slab_us(l.q.bm, f.out_type == DT_F32) + (l.direct ? 0.0 : staged_us(l.q.bm));
    double us = rounds_of(ceil_div(f.M, l.q.bm) * ceil_div(f.N, l.q.bn) * l.q.splits) * l.per_split * slab;
    if (l.q.splits > 1) us += kJoinUs + 2.0 * l.used / kBytesPerUs;
    if (l.copies) us += kJoinUs + 2.0 * (l.wants - l.used) / kBytesPerUs;
    return 2.7 + std::max(us, (double)f.N * f.K / 5.0e6);
}

hipError_t launch_f8_tile(const F8Params& f, void* ws, size_t ws_bytes, hipStream_t st) {
    const bool wide = f.out_type == DT_F32;
    if (!ws) ws_bytes = 0;
    F8Launch l = f8_launch_of(f, ws_bytes);
    const F8Plan& q = l.q;
    const bool copies = l.copies, direct = l.direct;
    const int64_t ldp = f8_ldp(f.N), kp = l.kp;
    const F8Extra x = {f.sa, f.sb, l.per_split, l.each};
    op_note("  %d x %d tiles, %d splits of K, %s loads%s", q.bm, q.bn, q.splits, direct ? "direct" : "staged", copies ? " of copied rows" : "");
    F8Params o = f;
    if (copies) {
        uint8_t* at = static_cast<uint8_t*>(ws) + l.used;
        RowsJob ja = {}, jb = {};
        if (l.copy_a) {
            ja = l.ja;
            o.A = ja.dst = at;
            o.lda = kp;
            at += ja.bytes();
        }
        if (l.copy_b) {
            jb = l.jb;
            o.B = jb.dst = at;
            o.ldb = kp;
        }
        const hipError_t e = launch_rows_pack(ja, jb, st);
        if (e != hipSuccess) return e;
        o.K = (int)kp;
    }
    GemmParams p = {};
    p.A = reinterpret_cast<const char*>(o.A);
    p.B = reinterpret_cast<const char*>(o.B);
    p.C = f.C;
    p.lda = o.lda; p.ldb = o.ldb; p.ldc = f.ldc;
    p.M = f.M; p.N = f.N; p.K = o.K;
    p.alpha = f.alpha; p.beta = f.beta;
    p.out_type = f.out_type;
    p.tiles_m = (int)ceil_div(f.M, q.bm);
    p.tiles_n = (int)ceil_div(f.N, q.bn);
    p.group_m = 8;
    p.xcd_remap = 1;
    if (q.splits > 1) {
        GemmParams s = p;
        F8Extra y = x;
        y.sa = y.sb = nullptr;
        s.C = static_cast<char*>(ws);
        s.ldc = ldp;
        s.alpha = 1.0f;
        s.beta = 0.0f;
        const hipError_t e = wide ? tile_of<DT_F32, true>(q, direct, s, y, st) : tile_of<DT_F32, false>(q, direct, s, y, st);
        if (e != hipSuccess) return e;
        if (wide) return join_of<DT_F32>(p, x, ws, ldp, q.splits, st);
        return f.out_type == DT_BF16 ? join_of<DT_BF16>(p, x, ws, ldp, q.splits, st) : join_of<DT_F16>(p, x, ws, ldp, q.splits, st);
    }
    if (wide) return tile_of<DT_F32, true>(q, direct, p, x, st);
    return f.out_type == DT_BF16 ? tile_of<DT_BF16, false>(q, direct, p, x, st) : tile_of<DT_F16, false>(q, direct, p, x, st);
}

}  // namespace gemm
