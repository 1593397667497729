// linear_grad.hip -- the products of the backward pass of gemm_linear, on tiles: C = A B with B (K x N) row by row and A either
// K-contiguous (dA = dZ W) or row by row too (dW = dZ^T A, A here the transpose that dZ is in memory).
//
// Neither is rewritten: an operand whose rows run along the sum is copied into LDS as it lies, 64 rows of the tile's columns, and
// read transposed, ds_read_b64_tr_b16: within 16 lanes, lane j points at row kb + j / 4, columns nb + 4 (j mod 4), and lane i
// receives rows kb .. kb + 3 of column nb + i.  Two of them make the eight k of a 16 x 16 x 32 instruction's lane.  A group of 16
// lanes reads 32 bytes of four rows, whose pitch is a multiple of the banks; so 32-byte piece q of row r lies at piece
// q ^ tr_swz(r), and the eight rows that 32 lanes read are apart.  Copies go straight to LDS, by the form that the compiler does not
// count as an LDS access (it would have every transposed read wait for all of them).
//
// What is left of K behind whole slabs of 64 is loaded through registers behind the loop, zeros where there is nothing.
// Where tiles do not fill the card the sum is split over workgroups, and a second launch adds the parts in order.
#include <algorithm>

#include "linear.hpp"
#include "linear_plan.hpp"
#include "rows_pack.hpp"

namespace gemm {
namespace {

// Row r's place for its 32-byte pieces, by width C: rows r, r + 1, r + 2, r + 3 and r + 16, ... r + 19 (r a multiple of 4) differ.
template <int C>
__device__ __forceinline__ int tr_swz(int r) {
    if constexpr (C == 64) return (r >> 1 & 1) | (r >> 4 & 1) << 1;   // (four pieces a row, two rows in the banks' width)
    else return (r & 3) | (r >> 4 & 1) << 2;
}
__device__ __forceinline__ void copy16(const char* base, uint32_t off, LDS_AS char* to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" :: "v"(off), "s"(base), "s"((uint32_t)(uintptr_t)to) : "m0");
}

// 64 rows of C columns, as they lie.  Columns from `cols` on (a multiple of 8) read the last eight again.
template <int C, int NW>
struct RowsOperand {
    static constexpr int ROWB = C * 2, CPR = ROWB / 16, RPI = 64 / CPR, IPW = 64 / (RPI * NW), NP = RPI < 4 ? 4 / RPI : 1;
    static_assert(IPW * RPI == 16, "sixteen rows a wave: the swizzle's high bit is the wave's");
    const char* base;
    int64_t step, ld;
    uint32_t pat[NP];
    int w, cols;
    __device__ __forceinline__ int chunk(int row, int pc) const { return pc ^ tr_swz<C>(row) << 1; }
    __device__ __forceinline__ void init(const char* origin, int64_t ld_bytes, int cols_) {
        base = origin;
        ld = ld_bytes;
        step = 64 * ld_bytes;
        cols = cols_;
        w = wave_id();
        const int lr = lane_id() / CPR, pc = lane_id() % CPR;
#pragma unroll
        for (int ph = 0; ph < NP; ++ph) {
            const int c = chunk(w * 16 + ph * RPI + lr, pc);
            pat[ph] = (uint32_t)lr * (uint32_t)ld_bytes + 16 * min(c, cols / 8 - 1);
        }
    }
    __device__ __forceinline__ void issue(int slab, LDS_AS char* tile, int i0, int i1) const {
        const char* g = base + slab * step;
#pragma unroll
        for (int i = 0; i < IPW; ++i)
            if (i >= i0 && i < i1) copy16(g + (uint32_t)((w * IPW + i) * RPI) * (uint32_t)ld, pat[i % NP], tile + (w * IPW + i) * 1024);
    }
    // The first `left` rows of a slab through registers, zeros below, by NT threads.
    template <int NT>
    __device__ __forceinline__ void tail(int slab, int left, LDS_AS char* tile) const {
        const char* g = base + slab * step;
#pragma unroll
        for (int i = 0; i < 64 * CPR / NT; ++i) {
            const int id = (int)threadIdx.x + i * NT, row = id / CPR, pc = id % CPR, c = chunk(row, pc);
            u32x4 v = {0u, 0u, 0u, 0u};
            if (row < left) v = *reinterpret_cast<const u32x4*>(g + row * ld + 16 * min(c, cols / 8 - 1));
            *reinterpret_cast<LDS_AS u32x4*>(tile + id * 16) = v;
        }
    }
};
// R rows of 64 columns along the sum; rows from `rows` on read the last again.
template <int R, int NW>
struct SumOperand {
    static constexpr int ROWB = 128, IPW = R / (8 * NW);
    const char* base;
    int64_t ld;
    uint32_t at[IPW];
    int w, rows;
    __device__ __forceinline__ void init(const char* origin, int64_t ld_bytes, int rows_) {
        base = origin;
        ld = ld_bytes;
        rows = rows_;
        w = wave_id();
#pragma unroll
        for (int i = 0; i < IPW; ++i) {
            const int row = (w * IPW + i) * 8 + lane_id() / 8, c = lane_id() % 8 ^ swz<8>(row);
            at[i] = (uint32_t)min(row, rows - 1) * (uint32_t)ld_bytes + 16 * c;
        }
    }
    __device__ __forceinline__ void issue(int slab, LDS_AS char* tile, int i0, int i1) const {
        const char* g = base + (int64_t)slab * 128;
#pragma unroll
        for (int i = 0; i < IPW; ++i)
            if (i >= i0 && i < i1) copy16(g, at[i], tile + (w * IPW + i) * 1024);
    }
    // The first `left` columns (whole chunks of 8: what they hold past K is zero).
    template <int NT>
    __device__ __forceinline__ void tail(int slab, int left, LDS_AS char* tile) const {
        const char* g = base + (int64_t)slab * 128;
#pragma unroll
        for (int i = 0; i < R * 8 / NT; ++i) {
            const int id = (int)threadIdx.x + i * NT, row = id / 8, c = id % 8 ^ swz<8>(row);
            u32x4 v = {0u, 0u, 0u, 0u};
            if (8 * c < left) v = *reinterpret_cast<const u32x4*>(g + (int64_t)min(row, rows - 1) * ld + 16 * c);
            *reinterpret_cast<LDS_AS u32x4*>(tile + id * 16) = v;
        }
    }
};

template <typename T, bool ROWS_A, int BM, int BN, int WM, int WN, int NC, bool COPY>
struct GradOps : MfmaCompute<T, BM, BN, 64, WM, WN, 16> {
    typedef MfmaCompute<T, BM, BN, 64, WM, WN, 16> C;
    typedef typename C::frag_t frag_t;
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    std::conditional_t<ROWS_A, RowsOperand<BM, NC>, SumOperand<BM, NC>> la;
    RowsOperand<BN, NC> lb;
    static constexpr int LA = decltype(la)::IPW, L = LA + decltype(lb)::IPW;
    static constexpr int READS = (ROWS_A ? 2 : 1) * C::TM + 2 * C::TN;   // of LDS in a step
    uint32_t ta[ROWS_A ? C::TM : 1], tb[C::TN];   // a lane's piece of fragment i, first four k of step 0

    __device__ __forceinline__ void init(LDS_AS char* smem_) {
        C::init(smem_);
        const int w = wave_id(), lane = lane_id(), g = lane / 16, j = lane % 16;
        const int r = 8 * ((g & 1) * 2 + (g >> 1)) + j / 4;   // (the k order of the K-contiguous operand)
        auto piece = [&](auto width, int q) {
            constexpr int W = decltype(width)::value;
            return (uint32_t)(r * W * 2 + ((q ^ tr_swz<W>(r)) << 5) + j % 4 * 8);
        };
        if constexpr (ROWS_A) {
#pragma unroll
            for (int i = 0; i < C::TM; ++i) ta[i] = piece(std::integral_constant<int, BM>{}, w / WN * C::TM + i);
        }
#pragma unroll
        for (int i = 0; i < C::TN; ++i) tb[i] = C::A_BYTES + piece(std::integral_constant<int, BN>{}, w % WN * C::TN + i);
    }
    template <int W>
    static __device__ __forceinline__ frag_t read_tr(LDS_AS const char* at) {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s16x4*)(at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s16x4*)(at + 4 * W * 2));
        return __builtin_bit_cast(frag_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    template <int BUF>
    __device__ __forceinline__ void frag(int, int slot, int ks) {
        LDS_AS const char* st = this->smem + slot * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::TM; ++i) {
            if constexpr (ROWS_A) this->fa[BUF][i] = read_tr<BM>(st + ta[i] + ks * 32 * BM * 2);
            else this->fa[BUF][i] = *reinterpret_cast<LDS_AS const frag_t*>(st + this->a_off[ks] + i * 16 * C::ROWB);
        }
#pragma unroll
        for (int i = 0; i < C::TN; ++i) this->fb[BUF][i] = read_tr<BN>(st + tb[i] + ks * 32 * BN * 2);
    }
    // The products of a step, the next one's LDS reads spread over the first of them.
    template <int BUF, int HAS, int PARTS>
    __device__ __forceinline__ void math(int) {
        constexpr int NM = C::TM * C::TN, PER = (READS + NM - 1) / NM;
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int j = 0; j < C::TN; ++j) this->acc[i][j] = Mfma<T, 16>::run(this->fb[BUF][j], this->fa[BUF][i], this->acc[i][j]);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                           // MFMA
            if (i * PER < READS) __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);    // DS read
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void issue(int slab, int slot, int part, int parts) {
        if (!COPY) return;
        LDS_AS char* st = this->smem + slot * C::STAGE;
        const int c0 = part * L / parts, c1 = (part + 1) * L / parts;
        la.issue(slab, st, c0, c1 < LA ? c1 : LA);
        lb.issue(slab, st + C::A_BYTES, c0 > LA ? c0 - LA : 0, c1 - LA);
    }
    template <int N>
    __device__ __forceinline__ void wait_slabs() { if (COPY) wait_vm<N * L>(); }
    __device__ __forceinline__ void wait_lds() { wait_lgkm0(); }
    __device__ __forceinline__ void barrier() { gemm::barrier(); }
    // What the sum has behind its whole slabs, once every wave is through with those.
    __device__ __forceinline__ void tail(int slab, int left) {
        constexpr int NT = 64 * WM * WN;
        wait_lgkm0();
        gemm::barrier();
        la.template tail<NT>(slab, left, this->smem);
        lb.template tail<NT>(slab, left, this->smem + C::A_BYTES);
        wait_lgkm0();
        gemm::barrier();
        frag<0>(0, 0, 0);
        if (left > 32) frag<1>(0, 0, 1);
        math<0, 0, 1>(0);
        if (left > 32) math<1, 0, 1>(1);
    }
};

struct GradSplit {
    int per;           // slabs of K per split
    int64_t each;      // bytes between the splits' sums (in C's place)
};

// Splits of K (blockIdx.y) store plain sums, each into its own place; the last one has what is left behind whole slabs.
template <int T, int OUT, bool ROWS_A, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2)))
void linear_grad_kernel(GemmParams p, const GradSplit x, int a_cols, int b_cols) {
    typedef half_of<T> H;
    constexpr int NW = WM * WN, NC = NW < 4 ? NW : 4, STAGE = (BM + BN) * 128;
    constexpr int EPI = (OUT != DT_F32 && BN == 256) ? BM * BN * 2 : 0;
    __shared__ __attribute__((aligned(1024))) char smem_raw[S * STAGE > EPI ? S * STAGE : EPI];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m_keep = tm * BM, n_keep = tn * BN;
    // edge tiles shifted inward; where there are fewer rows or columns than a tile has, the operands repeat their last
    const int m0 = max(0, min(m_keep, (ROWS_A ? a_cols : p.M) - BM)), n0 = max(0, min(n_keep, b_cols - BN));
    const int s0 = (int)blockIdx.y * x.per, whole = p.K / 64;
    const bool last = blockIdx.y + 1 == gridDim.y;
    const int slabs = last ? whole - s0 : x.per, left = last ? p.K % 64 : 0;
    const char* A = p.A + (ROWS_A ? ((int64_t)s0 * 64 * p.lda + m0) * 2 : ((int64_t)m0 * p.lda + (int64_t)s0 * 64) * 2);
    const char* B = p.B + ((int64_t)s0 * 64 * p.ldb + n0) * 2;
    p.C += blockIdx.y * x.each;
    auto run = [&](auto& ops) {
        ops.init(smem);
        ops.la.init(A, p.lda * 2, (ROWS_A ? a_cols : p.M) - m0);
        ops.lb.init(B, p.ldb * 2, b_cols - n0);
        gemm_sched::ring_mainloop<S, 2, 1>(ops, slabs);
        if (left > 0) ops.tail(slabs, left);
        if constexpr (EPI > 0) {
            if (m0 == m_keep && n0 == n_keep && m0 + BM <= p.M && n0 + BN <= p.N && (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 &&
                (p.ldc * 2) % 16 == 0) {
                ops.template epilogue_lds<OUT, 64 * NW>(p, m0, n0);
                return;
            }
        }
        ops.template epilogue<OUT>(p, m0, n0, m_keep, n_keep);
    };
    if (NC == NW || wave_id() < NC) {
        GradOps<H, ROWS_A, BM, BN, WM, WN, NC, true> ops;
        run(ops);
    } else if constexpr (NC < NW) {
        GradOps<H, ROWS_A, BM, BN, WM, WN, NC, false> ops;
        run(ops);
    }
}

// C = the splits' sums, added in order.
template <int OUT>
__global__ __launch_bounds__(256) void linear_grad_join_kernel(const GemmParams p, const char* part, int64_t each, int ldp, int splits) {
    const int64_t quads = ldp / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= quads * p.M) return;
    const int64_t m = id / quads;
    const int n = (int)(id % quads) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < splits; ++i) s += *reinterpret_cast<const f32x4*>(part + i * each + (m * ldp + n) * 4);
    store4<OUT>(p, m, n, s);
}

// 256 x 256, or 128 x 128 and (A along the sum) 64 x 128 with splits.
TilePlan grad_plan(int64_t M, int64_t N, int64_t K, int least) {
    const int64_t cu = num_compute_units();
    const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128), t256 = ceil_div(M, 256) * ceil_div(N, 256);
    if (M >= 256 && N >= 256 && ceil_div(t256, cu) * 4.0 <= ceil_div(t128, cu) * kSmallCost) return TilePlan{256, 256, 1};
    if (t128 > cu && M >= 128) return TilePlan{128, 128, 1};
    return small_plan(M, N, std::max<int64_t>(1, K / 64), M >= 128 || least == 128 ? 128 : 64, least, 64, (N + 7) / 8 * 8);
}

struct GradLaunch {
    TilePlan q;
    int per_split;
    int64_t each, ldp;
    RowsJob ja, jb;        // copies of what is not aligned, behind the splits' sums
    bool copy_a, copy_b;
    size_t used, wants;
};
GradLaunch launch_of(const GradParams& f, size_t ws_bytes) {
    GradLaunch l;
    l.q = grad_plan(f.M, f.N, f.K, f.rows_a ? 128 : 64);
    const int64_t slabs = std::max<int64_t>(1, f.K / 64);
    l.ldp = (f.N + 7) / 8 * 8;
    l.each = (int64_t)f.M * l.ldp * (int64_t)sizeof(float);
    // (an operand of the sum's length, or of the rows' or columns' that the tiles take eight at a time)
    const int64_t a_rows = f.rows_a ? f.K : f.M, a_len = f.rows_a ? f.M : f.K;
    l.copy_a = a_len % 8 || f.lda % 8 || (uintptr_t)f.A % 16;
    l.copy_b = f.N % 8 || f.ldb % 8 || (uintptr_t)f.B % 16;
    l.ja = {reinterpret_cast<const uint8_t*>(f.A), nullptr, f.lda * 2, a_rows, a_len * 2, a_rows, (a_len + 7) / 8 * 16};
    l.jb = {reinterpret_cast<const uint8_t*>(f.B), nullptr, f.ldb * 2, f.K, (int64_t)f.N * 2, f.K, ((int64_t)f.N + 7) / 8 * 16};
    const size_t copies = ((l.copy_a ? l.ja.bytes() : 0) + (l.copy_b ? l.jb.bytes() : 0) + 255) & ~size_t(255);
    const size_t room = ws_bytes > copies ? ws_bytes - copies : 0;
    if (l.q.splits > 1 && room < (size_t)(l.q.splits * l.each)) l.q.splits = (int)(room / l.each);
    if (l.q.splits < 2) l.q.splits = 1;
    l.per_split = (int)ceil_div(slabs, l.q.splits);
    l.q.splits = (int)ceil_div(slabs, l.per_split);
    l.used = copies;
    l.wants = copies + (l.q.splits > 1 ? (size_t)(l.q.splits * l.each) : 0);
    return l;
}

template <int T, int OUT, bool ROWS_A, int BM, int BN, int WM, int WN, int S>
hipError_t go(const GemmParams& p, const GradSplit& x, int splits, int a_cols, int b_cols, hipStream_t st) {
    hipLaunchKernelGGL((linear_grad_kernel<T, OUT, ROWS_A, BM, BN, WM, WN, S>), dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)splits),
                       dim3(64 * WM * WN), 0, st, p, x, a_cols, b_cols);
    return hipGetLastError();
}
template <int T, int OUT, bool ROWS_A>
hipError_t tile_of(const TilePlan& q, const GemmParams& p, const GradSplit& x, int a_cols, int b_cols, hipStream_t st) {
    if (q.bm == 256) return go<T, OUT, ROWS_A, 256, 256, 2, 4, 2>(p, x, q.splits, a_cols, b_cols, st);
    const bool alone = (int64_t)p.tiles_m * p.tiles_n * q.splits <= num_compute_units();
    if constexpr (!ROWS_A) {
        if (q.bm == 64)
            return alone ? go<T, OUT, ROWS_A, 64, 128, 2, 4, 4>(p, x, q.splits, a_cols, b_cols, st)
                         : go<T, OUT, ROWS_A, 64, 128, 2, 4, 2>(p, x, q.splits, a_cols, b_cols, st);
    }
    return alone ? go<T, OUT, ROWS_A, 128, 128, 2, 4, 4>(p, x, q.splits, a_cols, b_cols, st)
                 : go<T, OUT, ROWS_A, 128, 128, 2, 2, 2>(p, x, q.splits, a_cols, b_cols, st);
}

}  // namespace

// Strides whose offsets 32 bits hold, and room for copies of what is not aligned.
bool linear_grad_fits(const GradParams& f, size_t ws_bytes) {
    const int64_t most = int64_t(1) << 21;
    if (f.K < 1 || f.lda > most || f.ldb > most || f.K > most * 64 || (!f.rows_a && f.K > most)) return false;
    if (ceil_div(f.M, 64) * ceil_div(f.N, 128) >= (int64_t(1) << 22)) return false;
    const GradLaunch l = launch_of(f, ws_bytes);
    return l.used <= ws_bytes && l.used < (size_t(1) << 34) && (!l.copy_a || l.ja.len_pad / 2 <= most) && (!l.copy_b || l.jb.len_pad / 2 <= most);
}
size_t linear_grad_workspace(const GradParams& f) { return launch_of(f, SIZE_MAX / 2).wants; }

hipError_t launch_linear_grad(int in_type, const GradParams& f, void* ws, size_t ws_bytes, hipStream_t st) {
    const GradLaunch l = launch_of(f, ws_bytes);
    const TilePlan& q = l.q;
    op_note("  %d x %d x %d: %d x %d tiles, %d splits of the sum%s", f.M, f.N, f.K, q.bm, q.bn, q.splits, l.copy_a || l.copy_b ? ", of copied rows" : "");
    GemmParams p = {};
    p.A = f.A;
    p.B = f.B;
    p.C = f.C;
    p.lda = f.lda; p.ldb = f.ldb; p.ldc = f.ldc;
    p.M = f.M; p.N = f.N; p.K = f.K;
    p.alpha = 1.0f;
    p.tiles_m = (int)ceil_div(f.M, q.bm);
    p.tiles_n = (int)ceil_div(f.N, q.bn);
    p.group_m = 8;
    p.xcd_remap = 1;
    if (l.copy_a || l.copy_b) {
        uint8_t* at = static_cast<uint8_t*>(ws);
        RowsJob ja = {}, jb = {};
        if (l.copy_a) {
            ja = l.ja;
            ja.dst = at;
            p.A = reinterpret_cast<const char*>(at);
            p.lda = ja.len_pad / 2;
            at += ja.bytes();
        }
        if (l.copy_b) {
            jb = l.jb;
            jb.dst = at;
            p.B = reinterpret_cast<const char*>(at);
            p.ldb = jb.len_pad / 2;
        }
        const hipError_t e = launch_rows_pack(ja, jb, st);
        if (e != hipSuccess) return e;
    }
    const int a_cols = (f.M + 7) / 8 * 8, b_cols = (f.N + 7) / 8 * 8;
    const GradSplit x = {l.per_split, q.splits > 1 ? l.each : 0};
    GemmParams s = p;
    if (q.splits > 1) {
        s.C = static_cast<char*>(ws) + l.used;
        s.ldc = l.ldp;
    }
    auto tiles = [&](auto t, auto o) {
        constexpr int T = decltype(t)::value, OUT = decltype(o)::value;
        return f.rows_a ? tile_of<T, OUT, true>(q, s, x, a_cols, b_cols, st) : tile_of<T, OUT, false>(q, s, x, a_cols, b_cols, st);
    };
    const hipError_t e = by_type(in_type, q.splits > 1 ? (int)DT_F32 : f.out_type, tiles);
    if (e != hipSuccess || q.splits == 1) return e;
    return by_type(in_type, f.out_type, [&](auto, auto o) {
        hipLaunchKernelGGL((linear_grad_join_kernel<decltype(o)::value>), dim3((unsigned)ceil_div(f.M * (l.ldp / 4), 256)), dim3(256), 0, st, p,
                           s.C, l.each, (int)l.ldp, q.splits);
        return hipGetLastError();
    });
}

}  // namespace gemm
