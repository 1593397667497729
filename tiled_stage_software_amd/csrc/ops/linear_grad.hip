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
// 4096 x 14336 x 4096 bf16: dA 352 us, dW 390 (1.37 and 1.23 PFLOP/s; matrix cores 71% and 66% busy; dW's 896 tiles of 256 x 256 are three
// and a half rounds).  With operands rewritten ahead of them they took 542 and 482.
//
// Where tiles do not fill the card the sum is split over workgroups, and a second launch adds the parts in order.
#include <algorithm>

#include "linear.hpp"
#include "linear_plan.hpp"

namespace gemm {
namespace {

// Row r's place for its 32-byte pieces (rows of C columns): r, r + 1, r + 2, r + 3 and r + 16, ... r + 19 (r a multiple of 4) differ.
template <int C>
__device__ __forceinline__ int tr_swz(int r) {
    static_assert(C >= 128, "eight pieces a row");
    return (r & 3) | (r >> 4 & 1) << 2;
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

struct GradSide {     // one product
    GemmParams p;
    int per;           // slabs of K per split
    int64_t each;      // bytes between the splits' sums (in C's place)
    int a_cols, b_cols, splits;
    uint32_t blocks;
};

// Workgroup wg of a product.  Splits of K store plain sums, each into its own place; the last one has what is left behind whole
// slabs.  OUT: C's type (-1: as p.out_type says, T or fp32).
template <int T, int OUT, bool ROWS_A, int BM, int BN, int WM, int WN, int S>
__device__ __forceinline__ void grad_tile(const GradSide& x, uint32_t wg, LDS_AS char* smem) {
    typedef half_of<T> H;
    constexpr int NW = WM * WN, NC = NW < 4 ? NW : 4;
    GemmParams p = x.p;
    const int tiles = p.tiles_m * p.tiles_n, split = (int)(wg / (uint32_t)tiles);
    int tm, tn;
    tile_coords_of(p, (int)(wg - (uint32_t)split * (uint32_t)tiles), tm, tn);
    const int m_keep = tm * BM, n_keep = tn * BN;
    // edge tiles shifted inward; where there are fewer rows or columns than a tile has, the operands repeat their last
    const int a_end = ROWS_A ? x.a_cols : p.M;
    const int m0 = max(0, min(m_keep, a_end - BM)), n0 = max(0, min(n_keep, x.b_cols - BN));
    const int s0 = split * x.per, whole = p.K / 64;
    const bool last = split + 1 == x.splits;
    const int slabs = last ? whole - s0 : x.per, left = last ? p.K % 64 : 0;
    const char* A = p.A + (ROWS_A ? ((int64_t)s0 * 64 * p.lda + m0) * 2 : ((int64_t)m0 * p.lda + (int64_t)s0 * 64) * 2);
    const char* B = p.B + ((int64_t)s0 * 64 * p.ldb + n0) * 2;
    p.C += split * x.each;
    auto run = [&](auto& ops) {
        ops.init(smem);
        ops.la.init(A, p.lda * 2, a_end - m0);
        ops.lb.init(B, p.ldb * 2, x.b_cols - n0);
        gemm_sched::ring_mainloop<S, 2, 1>(ops, slabs);
        if (left > 0) ops.tail(slabs, left);
        if constexpr (OUT == T && BN == 256) {
            if (m0 == m_keep && n0 == n_keep && m0 + BM <= p.M && n0 + BN <= p.N && (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 &&
                (p.ldc * 2) % 16 == 0) {
                ops.template epilogue_lds<OUT, 64 * NW>(p, m0, n0);
                return;
            }
        }
        // (rows of any alignment in whole vectors)
        const LinearEpi e = {nullptr, nullptr, nullptr, p.C, 0, 0, p.ldc, p.M, p.N, 0, ACT_NONE};
        constexpr int BYTES = S * (BM + BN) * 128;
        if constexpr (OUT >= 0) {
            linear_epilogue<T, OUT, BM, BN, WM, WN, 16, BYTES>(ops, e, smem, m0, n0, m_keep, n_keep);
        } else {
            if (p.out_type == DT_F32) linear_epilogue<T, DT_F32, BM, BN, WM, WN, 16, BYTES>(ops, e, smem, m0, n0, m_keep, n_keep);
            else linear_epilogue<T, T, BM, BN, WM, WN, 16, BYTES>(ops, e, smem, m0, n0, m_keep, n_keep);
        }
    };
    if (NC == NW || wave_id() < NC) {
        GradOps<H, ROWS_A, BM, BN, WM, WN, NC, true> ops;
        run(ops);
    } else if constexpr (NC < NW) {
        GradOps<H, ROWS_A, BM, BN, WM, WN, NC, false> ops;
        run(ops);
    }
}
template <int T, int OUT, bool ROWS_A, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2)))
void linear_grad_kernel(const GradSide x) {
    constexpr int RING = S * (BM + BN) * 128, EPI = (OUT == T && BN == 256) ? BM * BN * 2 : 0;
    __shared__ __attribute__((aligned(1024))) char smem_raw[RING > EPI ? RING : EPI];
    grad_tile<T, OUT, ROWS_A, BM, BN, WM, WN, S>(x, blockIdx.x, (LDS_AS char*)smem_raw);
}
// Both products in one launch, where together they leave compute units empty.
template <int T, int BM>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2)))
void linear_grads_kernel(const GradSide a, const GradSide w) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[4 * 256 * 128];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    if (blockIdx.x < a.blocks) grad_tile<T, -1, false, BM, 128, 2, 4, 4>(a, blockIdx.x, smem);
    else grad_tile<T, -1, true, 128, 128, 2, 4, 4>(w, blockIdx.x - a.blocks, smem);
}

// The last launch: C = the splits' sums, added in order, of either product, and db = its parts' (64 columns a workgroup, every
// fourth part a wave).
struct JoinSide {
    GemmParams p;
    const char* part;
    int64_t each;
    int ldp, splits;
    uint32_t blocks;
};
__global__ __launch_bounds__(256) void linear_grad_join_kernel(const JoinSide a, const JoinSide w, const DbJoin d) {
    uint32_t block = blockIdx.x;
    if (block < a.blocks + w.blocks) {
        const bool second = block >= a.blocks;
        if (second) block -= a.blocks;
        const JoinSide& x = second ? w : a;
        const int64_t quads = x.ldp / 4, id = (int64_t)block * 256 + threadIdx.x;
        if (id >= quads * x.p.M) return;
        const int64_t m = id / quads;
        const int n = (int)(id % quads) * 4;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int i = 0; i < x.splits; ++i) s += *reinterpret_cast<const f32x4*>(x.part + i * x.each + (m * x.ldp + n) * 4);
        if (x.p.out_type == DT_F32) store4<DT_F32>(x.p, m, n, s);
        else if (x.p.out_type == DT_BF16) store4<DT_BF16>(x.p, m, n, s);
        else store4<DT_F16>(x.p, m, n, s);
        return;
    }
    block -= a.blocks + w.blocks;
    __shared__ float sums[4][64];
    const int64_t n = (int64_t)block * 64 + lane_id();
    const int wave = wave_id();
    float s = 0.0f;
    if (n < d.N) {
#pragma unroll 8
        for (int i = wave; i < d.parts; i += 4) s += d.part[(int64_t)i * d.N + n];
    }
    sums[wave][lane_id()] = s;
    __syncthreads();
    if (wave == 0 && n < d.N) d.db[n] = sums[0][lane_id()] + sums[1][lane_id()] + sums[2][lane_id()] + sums[3][lane_id()];
}

int64_t slabs_of(const GradParams& f) { return std::max<int64_t>(1, f.K / 64); }
int64_t ldp_of(const GradParams& f) { return ((int64_t)f.N + 7) / 8 * 8; }
int64_t each_of(const GradParams& f) { return (int64_t)f.M * ldp_of(f) * (int64_t)sizeof(float); }
int64_t tiles_of(const GradParams& f, int bm, int bn) { return ceil_div(f.M, bm) * ceil_div(f.N, bn); }
size_t sums_of(const GradParams& f, int64_t splits) { return splits > 1 ? (size_t)(splits * each_of(f) + 255) & ~size_t(255) : 0; }

template <int T, bool ROWS_A>
hipError_t alone_of(const GradParams& f, const GradSide& x, hipStream_t st) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(x.blocks), dim3(512), 0, st, x);
        return hipGetLastError();
    };
    if (f.bm == 256)
        return x.p.out_type == DT_F32 ? go(linear_grad_kernel<T, DT_F32, ROWS_A, 256, 256, 2, 4, 2>)
                                      : go(linear_grad_kernel<T, T, ROWS_A, 256, 256, 2, 4, 2>);
    const bool alone = x.blocks <= (uint32_t)num_compute_units();
    if constexpr (!ROWS_A) {
        if (f.bm == 64) return alone ? go(linear_grad_kernel<T, -1, ROWS_A, 64, 128, 2, 4, 4>) : go(linear_grad_kernel<T, -1, ROWS_A, 64, 128, 2, 4, 3>);
    }
    return alone ? go(linear_grad_kernel<T, -1, ROWS_A, 128, 128, 2, 4, 4>) : go(linear_grad_kernel<T, -1, ROWS_A, 128, 128, 2, 4, 2>);
}

}  // namespace

// Aligned operands whose strides' offsets 32 bits hold (the caller copies others).
bool linear_grad_fits(const GradParams& f) {
    const int64_t most = int64_t(1) << 21;
    const int along = f.rows_a ? f.M : f.K;
    return f.K >= 1 && f.lda <= most && f.ldb <= most && f.K <= most * 64 && tiles_of(f, 64, 128) < (int64_t(1) << 22) && along <= most;
}

// A small product's splits, the launch that joins them not counted: it is one for both.
double grad_us(int64_t cu, const GradParams& f, int bm, int splits) {
    return slabs_us(cu, bm, tiles_of(f, bm, bm == 256 ? 256 : 128) * splits, ceil_div(slabs_of(f), splits), DIRECT);
}
// Splits, which are fewer where as many would leave some empty.
int64_t splits_of(const GradParams& f, int splits) { return ceil_div(slabs_of(f), ceil_div(slabs_of(f), splits)); }
double sums_us(const GradParams& f, int splits) { return 2.0 * (double)sums_of(f, splits) / kBytesPerUs; }

void linear_grad_plan(GradParams (&f)[2], size_t ws_bytes) {
    // each for itself: the tile and splits that should be fastest
    const int64_t cu = num_compute_units();
    size_t left = ws_bytes;
    double alone = 0.0;
    int joins = 0;
    for (GradParams& x : f) {
        x.ws = 0;
        x.splits = 1;
        x.bm = x.bn = 128;
        if (!x.C) continue;
        double best = 0.0;
        auto take = [&](int bm, int s) {
            const double us = grad_us(cu, x, bm, s) + (s > 1 ? kJoinUs + sums_us(x, s) : 0.0);
            if (best > 0.0 && us >= best) return;
            best = us;
            x.bm = bm;
            x.bn = bm == 256 ? 256 : 128;
            x.splits = s;
        };
        if (x.M >= 256 && x.N >= 256) take(256, 1);
        for (int bm : {128, 64}) {
            if (bm == 64 && (x.rows_a || tiles_of(x, 64, 128) > 16 * cu)) continue;
            for (int s : kSplits)
                if (s == 1 || (2 * s <= slabs_of(x) + 1 && tiles_of(x, bm, 128) * (s - 1) <= 2 * cu && sums_of(x, splits_of(x, s)) <= left)) take(bm, s);
        }
        left -= sums_of(x, splits_of(x, x.splits));
        alone += best + 2.5;   // (a launch)
        joins += x.splits > 1;
    }
    if (joins == 2) alone -= kJoinUs;
    // or both in one launch, where together they fill the compute units once at most
    if (f[0].C && f[1].C) {
        const GradParams &a = f[0], &w = f[1];
        double best = alone;
        int bm_a = 0, sa = 1, sw = 1;
        for (int bm : {128, 64})
            for (int s0 : kSplits) {
                if ((s0 > 1 && 2 * s0 > slabs_of(a) + 1) || tiles_of(a, bm, 128) * s0 >= cu) break;
                for (int s1 : kSplits) {
                    if ((s1 > 1 && 2 * s1 > slabs_of(w) + 1) || sums_of(a, splits_of(a, s0)) + sums_of(w, splits_of(w, s1)) > ws_bytes || tiles_of(a, bm, 128) * s0 + tiles_of(w, 128, 128) * s1 > cu) break;
                    const double us = 2.5 + std::max(grad_us(cu, a, bm, s0), grad_us(cu, w, 128, s1)) + (s0 > 1 || s1 > 1 ? kJoinUs : 0.0) + sums_us(a, s0) + sums_us(w, s1);
                    if (us >= best) continue;
                    best = us;
                    bm_a = bm, sa = s0, sw = s1;
                }
            }
        if (bm_a) {
            f[0].bm = bm_a;
            f[0].bn = f[1].bm = f[1].bn = 128;
            f[0].splits = sa;
            f[1].splits = sw;
        }
    }
    for (GradParams& x : f)
        if (x.C) {
            x.splits = (int)splits_of(x, x.splits);
            x.ws = sums_of(x, x.splits);
        }
}

hipError_t launch_linear_grad(int in_type, const GradParams (&f)[2], const DbJoin& db, void* ws, hipStream_t st) {
    GradSide side[2] = {};
    JoinSide join[2] = {};
    char* at = static_cast<char*>(ws);
    for (int i = 0; i < 2; ++i) {
        const GradParams& q = f[i];
        if (!q.C) continue;
        GradSide& x = side[i];
        GemmParams& p = x.p;
        p.A = q.A;
        p.B = q.B;
        p.C = q.C;
        p.lda = q.lda; p.ldb = q.ldb; p.ldc = q.ldc;
        p.M = q.M; p.N = q.N; p.K = q.K;
        p.alpha = 1.0f;
        p.out_type = q.out_type;
        p.tiles_m = (int)ceil_div(q.M, q.bm);
        p.tiles_n = (int)ceil_div(q.N, q.bn);
        p.group_m = 8;
        p.xcd_remap = 1;
        x.per = (int)ceil_div(slabs_of(q), q.splits);
        x.a_cols = (q.M + 7) / 8 * 8;
        x.b_cols = (q.N + 7) / 8 * 8;
        x.splits = q.splits;
        x.blocks = (uint32_t)(p.tiles_m * p.tiles_n * q.splits);
        if (q.splits > 1) {
            JoinSide& j = join[i];
            j.p = p;
            j.part = p.C = at;
            j.each = x.each = each_of(q);
            j.ldp = (int)(p.ldc = ldp_of(q));
            j.splits = q.splits;
            j.blocks = (uint32_t)ceil_div(q.M * (ldp_of(q) / 4), 256);
            p.out_type = DT_F32;
            at += q.ws;
        }
    }
    hipError_t e = hipSuccess;
    const bool together = side[0].blocks && side[1].blocks && f[0].bm < 256 && f[1].bm < 256 && side[0].blocks + side[1].blocks <= (uint32_t)num_compute_units();
    auto both = [&](auto t) {
        constexpr int T = decltype(t)::value;
        const dim3 grid(side[0].blocks + side[1].blocks);
        if (f[0].bm == 64) hipLaunchKernelGGL((linear_grads_kernel<T, 64>), grid, dim3(512), 0, st, side[0], side[1]);
        else hipLaunchKernelGGL((linear_grads_kernel<T, 128>), grid, dim3(512), 0, st, side[0], side[1]);
        return hipGetLastError();
    };
    auto each = [&](auto t) {
        constexpr int T = decltype(t)::value;
        hipError_t s = hipSuccess;
        if (side[0].blocks) s = alone_of<T, false>(f[0], side[0], st);
        if (s == hipSuccess && side[1].blocks) s = alone_of<T, true>(f[1], side[1], st);
        return s;
    };
    typedef std::integral_constant<int, DT_BF16> B;
    typedef std::integral_constant<int, DT_F16> H;
    if (together) e = in_type == DT_BF16 ? both(B{}) : both(H{});
    else e = in_type == DT_BF16 ? each(B{}) : each(H{});
    const uint32_t db_blocks = db.db ? (uint32_t)ceil_div(db.N, 64) : 0, blocks = join[0].blocks + join[1].blocks + db_blocks;
    if (e != hipSuccess || blocks == 0) return e;
    hipLaunchKernelGGL(linear_grad_join_kernel, dim3(blocks), dim3(256), 0, st, join[0], join[1], db);
    return hipGetLastError();
}

}  // namespace gemm
