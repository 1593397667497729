// linear_tile.hip -- the product with bias, activation and residual on tiles: BM x BN of C per workgroup, slabs of 64 of K in
// an LDS ring, v_mfma_f32_16x16x32 on 16 x 16 blocks.
//
// The ring, its loaders and the multiplication are those of the library's 16-bit products; what is new is the epilogue.  Tiles
// of 256 x 256 and 192 x 256 (eight waves, copies by one wave of each SIMD) for large products; 128 x 128 and 64 x 128, with
// K split over workgroups, where those leave the card empty.  What K has behind whole slabs is loaded through registers behind the
// loop.  Rows that the direct copies cannot take (not 16-byte aligned) are copied into the workspace first where that
// pays, or loaded through registers.
//
// Matrix cores bound large products, at the clock that the card's power leaves (bf16): 4096 x 4096 x 14336 with a residual 371 us (1.30
// PFLOP/s, matrix cores 65% busy, one round of 256 tiles), 8192 x 14336 x 4096 with gelu and Z 786 us (1.22; the sums alone 725: gelu and
// the second 16-bit result are 25 to 30 each, seven epilogues in turn on every compute unit).  Small ones are bound by a slab's way
// from the caches to LDS (linear_plan.hpp).  The epilogue turns the accumulators in LDS in fp32, so that a thread has eight
// neighbouring columns: whole loads and stores, one rounding.  Applied to the accumulators in registers instead it
// spilled them (850 us instead of 776).
#include <algorithm>

#include "f8_common.hpp"
#include "linear.hpp"
#include "linear_plan.hpp"
#include "rows_pack.hpp"
#include "short_loader.hpp"

namespace gemm {
namespace {

constexpr int kSlabBytes = 128, kSlab = 64;

// Direct global -> LDS copies by the first NC waves: 16-byte aligned rows, whole slabs and tiles.
template <typename T, int BM, int BN, int WM, int WN, int NC, bool COPY>
struct LinearRingOps : MfmaCompute<T, BM, BN, kSlab, WM, WN, 16> {
    typedef MfmaCompute<T, BM, BN, kSlab, WM, WN, 16> C;
    ALoader<BM, kSlabBytes, NC> la;
    DirectLoader<BN, kSlabBytes, NC, true> lb;
    static constexpr int LA = decltype(la)::IPW, L = LA + decltype(lb)::IPW;
    int first = 0, slabs = 0;   // small tiles take slab `first` first, and slab 0 behind the last
    __device__ __forceinline__ void issue(int slab, int slot, int part, int parts) {
        if (!COPY) return;
        if constexpr (BM <= 128) {
            slab += first;
            if (slab >= slabs) slab -= slabs;
        }
        LDS_AS char* st = this->smem + slot * C::STAGE;
        const int c0 = part * L / parts, c1 = (part + 1) * L / parts;
        la.issue(slab, st, c0, c1 < LA ? c1 : LA);
        lb.issue(slab, st + C::A_BYTES, c0 > LA ? c0 - LA : 0, c1 - LA);
    }
    template <int N>
    __device__ __forceinline__ void wait_slabs() { if (COPY) wait_vm<N * L>(); }
    __device__ __forceinline__ void wait_lds() { wait_lgkm0(); }
    __device__ __forceinline__ void barrier() { gemm::barrier(); }
    template <int BUF>
    __device__ __forceinline__ void frag(int, int slot, int ks) { C::template frag<BUF>(slot, ks); }
    template <int BUF, int HAS, int PARTS>
    __device__ __forceinline__ void math(int) { C::template math<BUF, (COPY && HAS) ? (L + PARTS - 1) / PARTS : 0>(); }
    // The last `bytes` (fewer than a slab's) of rows that begin at A and W, once every wave is through with the slabs; zeros behind
    // them, and the last row again where there are no more.
    __device__ __forceinline__ void tail(const char* A, int64_t lda, int a_rows, const char* W, int64_t ldw, int w_rows, int bytes) {
        constexpr int NT = 64 * WM * WN;
        wait_lgkm0();
        gemm::barrier();
#pragma unroll
        for (int i = 0; i < (BM + BN) * 8 / NT; ++i) {
            const int id = (int)threadIdx.x + i * NT, row = id / 8, c = id % 8;
            const char* at = row < BM ? A + (int64_t)min(row, a_rows - 1) * lda : W + (int64_t)min(row - BM, w_rows - 1) * ldw;
            const u32x4 v = load_chunk(reinterpret_cast<const uint8_t*>(at), 16 * c, bytes);
            *reinterpret_cast<LDS_AS u32x4*>(this->smem + row * kSlabBytes + ((c ^ swz<8>(row)) << 4)) = v;
        }
        wait_lgkm0();
        gemm::barrier();
        C::template frag<0>(0, 0);
        C::template frag<1>(0, 1);
        C::template math<0, 0>();
        C::template math<1, 0>();
    }
};

// Any pitch, alignment and K >= 64: 16-byte loads of any alignment into registers, two slabs ahead, written into the other
// slot under the first half of a slab's products.  A last slab that K does not fill is the row's last 128 bytes, with zeros in
// A and in W for what earlier slabs had (an infinity there times a zero would be NaN).  Rows past the end repeat the last.
template <typename T, int BM, int BN, int WM, int WN>
struct LinearStagedOps : MfmaCompute<T, BM, BN, kSlab, WM, WN, 16> {
    typedef MfmaCompute<T, BM, BN, kSlab, WM, WN, 16> C;
    static constexpr int NT = 64 * WM * WN, STEP = NT / 8;
    static constexpr int CA = BM / STEP, CH = (BM + BN) / STEP;   // chunks per thread and slab
    static_assert(BM % STEP == 0 && BN % STEP == 0 && STEP % 16 == 0, "rows split evenly; one swizzle phase per thread");
    static_assert(C::KS == 2, "a slab is two steps");
    const char* base[2];
    uint32_t off[CH], dst;
    u32x4 v[2][CH], mask = {~0u, ~0u, ~0u, ~0u};
    int64_t K;          // bytes of this workgroup's part of the rows
    __device__ __forceinline__ void init_rows(const char* A, int64_t lda, int m0, int M, const char* W, int64_t ldw, int n0, int N) {
        const int row = (int)threadIdx.x / 8, c = (int)threadIdx.x % 8;
        base[0] = A + (int64_t)m0 * lda;
        base[1] = W + (int64_t)n0 * ldw;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            off[i] = (i < CA ? (uint32_t)min(row + i * STEP, M - 1 - m0) * (uint32_t)lda
                             : (uint32_t)min(row + (i - CA) * STEP, N - 1 - n0) * (uint32_t)ldw) + 16 * c;
        dst = (uint32_t)(row * kSlabBytes + ((c ^ swz<8>(row)) << 4));
    }
    template <int V>
    __device__ __forceinline__ void load(int slab) {
        int64_t k = (int64_t)slab * kSlabBytes;
        if (k + kSlabBytes > K) {
            const int old = (int)(k + kSlabBytes - K) - (int)threadIdx.x % 8 * 16;   // bytes of this chunk that earlier slabs had
            k = K - kSlabBytes;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int o = old - 4 * q;
                mask[q] = o >= 4 ? 0u : o <= 0 ? ~0u : ~0u << (8 * o);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) v[V][i] = load16(base[i >= CA] + k + off[i]);
    }
    template <int V>
    __device__ __forceinline__ void put(int slot, bool last) {   // (the mask is the last slab's)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            u32x4 x = v[V][i];
            if (last) x &= mask;
            *reinterpret_cast<LDS_AS u32x4*>(this->smem + slot * C::STAGE + dst + i * STEP * kSlabBytes) = x;
        }
    }
    // Multiplies slab kt out of its slot, kt mod 2.  Slab kt + 2 is loaded into registers V; slab kt + 1 goes from registers W to the
    // other slot, which the barrier before this slab freed.
    template <int V, int W, bool LAST>
    __device__ __forceinline__ void slab(int kt, int slabs) {
        const int slot = kt & 1;
        C::template frag<1>(slot, 1);
        C::template math<0, 0>();
        if constexpr (!LAST) {
            put<W>(slot ^ 1, kt + 2 == slabs);
            load<V>(min(kt + 2, slabs - 1));
            wait_lgkm0();
            gemm::barrier();
            C::template frag<0>(slot ^ 1, 0);
        }
        C::template math<1, 0>();
    }
    __device__ __forceinline__ void run(int slabs) {
        load<0>(0);
        load<1>(min(1, slabs - 1));
        put<0>(0, slabs == 1);
        wait_lgkm0();
        gemm::barrier();
        C::template frag<0>(0, 0);
        int kt = 0;
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
};

struct LinearSplit {
    int per;           // slabs of K per split
    char* part;        // the splits' sums (NULL: there is one split, and the epilogue follows)
    int64_t each;      // bytes of a split's
};

// Columns of small tiles start a slab apart in K.  Workgroups run side by side, and where W's pitch is a power of two all of them would read
// the same few lines of every row at a time, which lie in few of the memory's channels: 64 x 14336 x 4096 34.8 us instead of 28.5, 128 rows
// 37.0 and 34.2.  Large tiles are not bound by W's bytes (no difference).
// S: slots of the ring (0: loads through registers, two slots).  Splits of K (blockIdx.y) store plain sums.
template <int T, int OUT, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2)))
void linear_tile_kernel(GemmParams p, const LinearEpi e, const LinearSplit x) {
    constexpr int NW = WM * WN, NC = NW < 4 ? NW : 4;
    constexpr int BYTES = (S > 0 ? S : 2) * (BM + BN) * kSlabBytes;
    __shared__ __attribute__((aligned(1024))) char smem_raw[BYTES];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m_keep = tm * BM, n_keep = tn * BN;
    const int m0 = max(0, min(m_keep, p.M - BM)), n0 = max(0, min(n_keep, p.N - BN));
    const int s0 = (int)blockIdx.y * x.per;
    const int64_t left = 2 * (int64_t)p.K - (int64_t)s0 * kSlabBytes, K = min(left, (int64_t)x.per * kSlabBytes);
    const int slabs = S > 0 ? (int)(K / kSlabBytes) : (int)((K + kSlabBytes - 1) / kSlabBytes);
    const char* A = p.A + (int64_t)s0 * kSlabBytes;
    const char* W = p.B + (int64_t)s0 * kSlabBytes;
    auto finish = [&](auto& ops) {
        if (x.part) {
            p.C = x.part + blockIdx.y * x.each;
            ops.template epilogue<DT_F32>(p, m0, n0, m_keep, n_keep);
        } else {
            linear_epilogue<T, OUT, BM, BN, WM, WN, 16, BYTES>(ops, e, smem, m0, n0, m_keep, n_keep);
        }
    };
    auto behind = [&](auto& ops) {
        const int bytes = (int)(K - (int64_t)slabs * kSlabBytes);
        if (bytes > 0)
            ops.tail(A + (int64_t)m0 * p.lda * 2 + (int64_t)slabs * kSlabBytes, p.lda * 2, p.M - m0, W + (int64_t)n0 * p.ldb * 2 + (int64_t)slabs * kSlabBytes,
                     p.ldb * 2, p.N - n0, bytes);
    };
    if constexpr (S > 0) {
        constexpr int KS = MfmaCompute<half_of<T>, BM, BN, kSlab, WM, WN, 16>::KS;
        if (NC == NW || wave_id() < NC) {
            LinearRingOps<half_of<T>, BM, BN, WM, WN, NC, true> ops;
            ops.init(smem);
            init_a<BM, kSlabBytes, NC>(ops.la, A + (int64_t)m0 * p.lda * 2, p.lda * 2, kSlabBytes, p.M - m0);
            ops.lb.init(W + (int64_t)n0 * p.ldb * 2, p.ldb * 2, kSlabBytes);
            if constexpr (BM <= 128) ops.slabs = slabs, ops.first = slabs > 0 ? tn % slabs : 0;
            gemm_sched::ring_mainloop<S, KS, 1>(ops, slabs);
            behind(ops);
            finish(ops);
        } else if constexpr (NC < NW) {
            LinearRingOps<half_of<T>, BM, BN, WM, WN, NC, false> ops;
            ops.init(smem);
            gemm_sched::ring_mainloop<S, KS, 1>(ops, slabs);
            behind(ops);
            finish(ops);
        }
    } else {
        LinearStagedOps<half_of<T>, BM, BN, WM, WN> ops;
        ops.init(smem);
        ops.init_rows(A, p.lda * 2, m0, p.M, W, p.ldb * 2, n0, p.N);
        ops.K = K;
        ops.run(slabs);
        finish(ops);
    }
}

// The epilogue of the splits' sums, added in order: eight columns of a row a thread.
template <int T, int OUT>
__global__ __launch_bounds__(256) void linear_join_kernel(const LinearEpi e, const LinearSplit x, int ldp, int splits) {
    const int64_t eights = ldp / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= eights * e.M) return;
    const int64_t m = id / eights;
    const int n = (int)(id % eights) * 8;
    float bias[8], v[8];
    load_bias<T>(e, n, bias);
    Eight<OUT> old;
    if (e.R) old.load(e.R + m * e.ldr * Elem<OUT>::SIZE, n, e.N);
    f32x4 s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
    for (int i = 0; i < splits; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[h] += *reinterpret_cast<const f32x4*>(x.part + i * x.each + (m * ldp + n + 4 * h) * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s[i / 4][i % 4];
    finish8<T, OUT>(e, m, n, 0, v, bias, old);
}

int64_t ldp_of(int64_t N) { return (N + 7) / 8 * 8; }

// What a call does with the workspace it has.
struct LinearLaunch {
    TilePlan q;          // 256 x 256, 192 x 256, 128 x 128 or 64 x 128
    int per_split;       // slabs of a split
    int64_t each;        // bytes of a split's sums
    RowsJob ja, jw;      // copies of the operands, behind the splits' sums ...
    bool copy_a, copy_w; // ... of those that the direct copies cannot take
    size_t used, wants;
    bool copies, direct;
};
constexpr size_t kMostCopied = size_t(1) << 34;   // rows_pack counts chunks in 32 bits

LinearLaunch with(const LinearParams& f, const TilePlan& q) {
    const int64_t slabs = ceil_div(f.K, kSlab), kp = (int64_t)(f.K + 7) / 8 * 16;
    LinearLaunch l = {};
    l.q = q;
    l.each = (int64_t)f.M * ldp_of(f.N) * (int64_t)sizeof(float);
    l.per_split = (int)ceil_div(slabs, q.splits);
    l.q.splits = (int)ceil_div(slabs, l.per_split);
    const int64_t least_a = least_rows(q.bm), least_w = q.bn;
    l.ja = {reinterpret_cast<const uint8_t*>(f.A), nullptr, f.lda * 2, f.M, (int64_t)f.K * 2, std::max<int64_t>(f.M, least_a), kp};
    l.jw = {reinterpret_cast<const uint8_t*>(f.W), nullptr, f.ldw * 2, f.N, (int64_t)f.K * 2, std::max<int64_t>(f.N, least_w), kp};
    l.copy_a = f.M < least_a || ((uintptr_t)f.A | (uint64_t)f.lda * 2) % 16;
    l.copy_w = f.N < least_w || ((uintptr_t)f.W | (uint64_t)f.ldw * 2) % 16;
    l.used = l.q.splits > 1 ? ((size_t)(l.q.splits * l.each) + 255) & ~size_t(255) : 0;
    l.wants = l.used + (l.copy_a ? l.ja.bytes() : 0) + (l.copy_w ? l.jw.bytes() : 0);
    l.direct = !l.copy_a && !l.copy_w;
    return l;
}
// The tile, the splits and the way of loading that should be fastest.
LinearLaunch launch_of(const LinearParams& f, size_t ws_bytes) {
    const int64_t slabs = ceil_div(f.K, kSlab), cu = num_compute_units();
    LinearLaunch best = {};
    double best_us = 0.0;
    for (int bm : {256, 192, 128, 64}) {
        const bool large = bm > 128;   // (no loads through registers, and no splits: small tiles fill the card better)
        const int bn = large ? 256 : 128;
        if (large && (f.M < bm || f.N < bn)) continue;
        const int64_t tiles = ceil_div(f.M, bm) * ceil_div(f.N, bn);
        if (bm == 64 && tiles > 16 * cu) continue;
        for (int s : kSplits) {
            if (s > 1 && (large || tiles > 2 * cu || s > 16 || s * 4 > slabs + 3 || tiles * s > 4 * cu)) break;
            LinearLaunch l = with(f, TilePlan{bm, bn, s});
            if (l.used > ws_bytes) break;
            const double copied = kCopyUs + 2.0 * (double)(l.wants - l.used) / kCopiedPerUs;
            const double staged = slabs_us(cu, bm, tiles * l.q.splits, l.per_split, STAGED);
            double us = slabs_us(cu, bm, tiles * l.q.splits, l.per_split, DIRECT);
            if (!l.direct) {
                l.copies = l.wants <= ws_bytes && l.wants < kMostCopied && (large || us + copied < staged);
                if (large && !l.copies) continue;
                us = l.copies ? us + copied : staged;
                l.direct = l.copies;
            }
            if (l.q.splits > 1) us += kJoinUs + 2.0 * (double)l.used / kBytesPerUs;
            if (best_us > 0.0 && us >= best_us) continue;
            best_us = us;
            best = l;
        }
    }
    return best;
}

template <int T, int OUT, int BM, int BN, int WM, int WN, int S>
hipError_t go(const GemmParams& p, const LinearEpi& e, const LinearSplit& x, int splits, hipStream_t st) {
    hipLaunchKernelGGL((linear_tile_kernel<T, OUT, BM, BN, WM, WN, S>), dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)splits),
                       dim3(64 * WM * WN), 0, st, p, e, x);
    return hipGetLastError();
}
// Small tiles that have a compute unit to themselves: four slots, so that three slabs are on their way.  Else a second workgroup, which
// fewer slots leave room for, hides the waits (eight waves either way: four measured 52.6 us instead of 48.4 on 264 tiles of 128 rows).
template <int T, int OUT>
hipError_t tile_of(const TilePlan& q, bool direct, const GemmParams& p, const LinearEpi& e, const LinearSplit& x, hipStream_t st) {
    if (q.bm == 256) return go<T, OUT, 256, 256, 2, 4, 2>(p, e, x, q.splits, st);
    if (q.bm == 192) return go<T, OUT, 192, 256, 2, 4, 2>(p, e, x, q.splits, st);
    const bool alone = (int64_t)p.tiles_m * p.tiles_n * q.splits <= num_compute_units();
    if (q.bm == 64) {
        if (!direct) return go<T, OUT, 64, 128, 2, 4, 0>(p, e, x, q.splits, st);
        return alone ? go<T, OUT, 64, 128, 2, 4, 4>(p, e, x, q.splits, st) : go<T, OUT, 64, 128, 2, 4, 3>(p, e, x, q.splits, st);
    }
    if (!direct) return go<T, OUT, 128, 128, 2, 4, 0>(p, e, x, q.splits, st);
    return alone ? go<T, OUT, 128, 128, 2, 4, 4>(p, e, x, q.splits, st) : go<T, OUT, 128, 128, 2, 4, 2>(p, e, x, q.splits, st);
}

}  // namespace

// K >= 64 and strides that the tiles' 32-bit offsets hold (256 rows below 2^31 bytes).
bool linear_tile_fits(const LinearParams& f) {
    const int64_t most = int64_t(1) << 21;
    return f.K >= kSlab && f.K <= most && f.lda <= most && f.ldw <= most && ceil_div(f.M, 64) * ceil_div(f.N, 128) < (int64_t(1) << 22);
}

size_t linear_tile_workspace(const LinearParams& f) {
    const LinearLaunch l = launch_of(f, SIZE_MAX / 2);
    return l.copies ? l.wants : l.used;
}

hipError_t launch_linear_tile(int in_type, const LinearParams& f, void* ws, size_t ws_bytes, hipStream_t st) {
    if (!ws) ws_bytes = 0;
    const LinearLaunch l = launch_of(f, ws_bytes);
    const TilePlan& q = l.q;
    op_note("  %d x %d tiles, %d splits of K, %s loads%s", q.bm, q.bn, q.splits, l.direct ? "direct" : "staged", l.copies ? " of copied rows" : "");
    GemmParams p = {};
    p.A = f.A;
    p.B = f.W;
    p.lda = f.lda; p.ldb = f.ldw;
    p.M = f.M; p.N = f.N; p.K = f.K;
    p.alpha = 1.0f;
    p.tiles_m = (int)ceil_div(f.M, q.bm);
    p.tiles_n = (int)ceil_div(f.N, q.bn);
    p.group_m = 8;
    p.xcd_remap = 1;
    if (l.copies) {
        uint8_t* at = static_cast<uint8_t*>(ws) + l.used;
        RowsJob ja = {}, jw = {};
        const int64_t kp = l.ja.len_pad / 2;
        if (l.copy_a) {
            ja = l.ja;
            ja.dst = at;
            p.A = reinterpret_cast<const char*>(at);
            p.lda = kp;
            at += ja.bytes();
        }
        if (l.copy_w) {
            jw = l.jw;
            jw.dst = at;
            p.B = reinterpret_cast<const char*>(at);
            p.ldb = kp;
        }
        const hipError_t e = launch_rows_pack(ja, jw, st);
        if (e != hipSuccess) return e;
    }
    const LinearEpi e = epi_of(f);
    LinearSplit x = {l.per_split, nullptr, l.each};
    const int64_t ldp = ldp_of(f.N);
    if (q.splits > 1) {
        x.part = static_cast<char*>(ws);
        p.ldc = ldp;
    }
    return by_type(in_type, f.out_type, [&](auto t, auto o) {
        constexpr int T = decltype(t)::value, OUT = decltype(o)::value;
        const hipError_t s = tile_of<T, OUT>(q, l.direct, p, e, x, st);
        if (s != hipSuccess || q.splits == 1) return s;
        hipLaunchKernelGGL((linear_join_kernel<T, OUT>), dim3((unsigned)ceil_div(f.M * (ldp / 8), 256)), dim3(256), 0, st, e, x, (int)ldp, q.splits);
        return hipGetLastError();
    });
}

}  // namespace gemm
