// w4_tile.hip -- the product with 4-bit weights on large tiles: BM x 128 of C per workgroup, four waves
// of BM x 32, slabs of 64 k in an LDS ring, v_mfma_f32_16x16x32 on 16 x 16 blocks.
//
// No weight is rounded, so a group's scale multiplies an fp32 sum: each accumulator has a second one
// for the running group, and an FMA for each joins them at the group's end.  That and
// turning codes into operands is vector work beside the matrix cores' (per wave, 128 x 32 tile and
// 128 k: 1024 cycles of matrix instructions; 4 x 2 x 8 operations for the codes, 64 for a group's end,
// four cycles each).  Wide blocks of A's rows keep it below theirs: one turned code serves BM / 16
// instructions (waves of 64 x 64, with half the fragment reads: 308 us instead of 300 for
// 2048 x 14336 x 4096; 96 rows and three workgroups a compute unit: 308; measured back to back, in turn with
// other work 261).  Groups shorter than 64 end with every 32 k (347 us).
//
// What the zero points take off a group is (1 + z/16) * (sum of A over it).  EACH: it comes off the group's dot product before
// the scale, a second FMA, so that the running sum over K never holds more than the result and one group.  For an fp32 C.
// Otherwise the part of all groups, sum over units of (s * (1 + z/16)) * (sum of A over the unit), is a product of its own
// with one k for a unit (a group; 32 k for short groups), and runs behind the loop on matrix instructions: 260 us instead of
// 275 (groups of 32: 347 and 371).  The running sum then holds what does not cancel until the end: on 300 x 4096 x 4096 and
// 14336 in f16, with a mean of three deviations in A, fp32 sums are off by 2.4e-5 and 5.0e-5 of the result instead of 3.1e-6
// (without a mean 9e-7 and 4e-7).  A 16-bit C's rounding hides that: 2.09e-4 and 2.13e-4 off in f16, of which the rounding is 2.08e-4.
//
// A launch before prepares the sums of A, in the order of the accumulators, and the scales and zero points, transposed to rows
// of columns; the ring brings along with the slabs what their ends need.
#include <algorithm>

#include "rows_pack.hpp"
#include "short_loader.hpp"
#include "w4_common.hpp"

namespace gemm {
namespace {

constexpr int kSlabK = 64, kBN = 128, kNC = 4;   // kNC: waves, side by side along N

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct W4Tile {
    GemmParams g;          // A, C, sizes, tiles; B unused
    const uint8_t* W;
    int64_t ldw;
    const char* sums;      // [unit][tile of M][BM] floats, a lane's together
    const char* scales;    // [unit][tile of N][128] floats, behind the sums
    const char* zeros;     // the same, behind the scales: -(1 + z/16) with EACH, -s * (1 + z/16) without
    int per_unit;          // slabs of a unit (0: two units to a slab)
    int per_split;         // slabs of a split of K
    int64_t part;          // bytes between the splits' results
};

// A row's two chunks of codes change places in every other eight rows, so that the 16 rows a read takes lie on
// different banks.
__device__ __forceinline__ int codes_swz(int row) { return (row >> 3) & 1; }

// S1: units are 32 k, two to a slab.  EACH: the zero points come off at each unit's end (the other form: zero_points()).
template <int T, int BM, bool S1, bool EACH>
struct W4Compute : MfmaCompute<typename Half<T>::type, BM, kBN, 64, 1, kNC, 16> {
    typedef MfmaCompute<typename Half<T>::type, BM, kBN, 64, 1, kNC, 16> C;
    static constexpr int TM = C::TM, TN = C::TN, AH = TM / 2, NU = S1 ? 2 : 1;
    static constexpr int A_BYTES = BM * 128, Q_BYTES = kBN * 32, S_AT = A_BYTES + Q_BYTES;
    static constexpr int SL = 8 * NU, RL = BM / 16;   // chunks of a wave's scales, [unit][8]; of a unit's sums that a wave copies
    static constexpr int UL = EACH ? 2 * SL + NU * RL : SL;   // of a wave: scales, then zero points, then its part of the sums
    static constexpr int STAGE = S_AT + kNC * UL * 16;
    static constexpr int KS = 4;   // steps of a slab: two k-steps by two halves of A's blocks
    static_assert(TN == 2 && TM % 2 == 0, "waves of 32 columns");
    f32x4 dot[TM][TN];
    u32x4 fa[2][AH], b[TN];
    uint32_t word[TN];
    f32x4 scale[TN], point[TN], a_sum[TM / 4];   // of the unit that ends next: scales, zero points, sums of A
    uint32_t qo, so, mo;   // LDS offsets of codes, scales and sums within a slot
    Spread<T> spread;
    int pos = 0, per_unit, left;   // slab within its unit; slabs left

    __device__ __forceinline__ void init(LDS_AS char* smem_, const W4Tile& p, int slabs) {
        C::init(smem_);
        const int wn = wave_id(), lane = lane_id(), r = lane % 16, g = lane / 16;
        const int kc = (g & 1) * 2 + (g >> 1);   // the k-chunk of lane group g, as in A's fragments
        qo = (uint32_t)(A_BYTES + (wn * 32 + r) * 32 + codes_swz(r) * 16 + kc * 4);
        so = (uint32_t)(S_AT + wn * UL * 16 + g * 16);
        const int at = r * TM / 4;   // this lane's sums, TM of them
        mo = (uint32_t)(S_AT + (at / RL * UL + 2 * SL + at % RL) * 16);
        per_unit = p.per_unit;
        left = slabs;
    }
    // Step q: half q % 2 of A's blocks at k-step q / 2, with the codes of the k-step.
    template <int BUF>
    __device__ __forceinline__ void frag(int, int slot, int q) {
        LDS_AS const char* st = this->smem + slot * STAGE;
#pragma unroll
        for (int i = 0; i < AH; ++i)
            fa[BUF][i] = *reinterpret_cast<LDS_AS const u32x4*>(st + this->a_off[q / 2] + (q % 2 * AH + i) * 16 * 128);
        if (q % 2 == 0) {
#pragma unroll
            for (int j = 0; j < TN; ++j) word[j] = *reinterpret_cast<LDS_AS const uint32_t*>(st + (qo ^ (q / 2 * 16)) + j * 16 * 32);
        }
        if (S1 ? q % 2 == 1 : q == 1) {   // (before the barrier that frees the slot)
            const int u = S1 ? q / 2 : 0;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                scale[j] = *reinterpret_cast<LDS_AS const f32x4*>(st + so + u * 128 + j * 64);
                if constexpr (EACH) point[j] = *reinterpret_cast<LDS_AS const f32x4*>(st + so + SL * 16 + u * 128 + j * 64);
            }
            if constexpr (EACH) {
#pragma unroll
                for (int i = 0; i < TM / 4; ++i) a_sum[i] = *reinterpret_cast<LDS_AS const f32x4*>(st + mo + (u * RL + i) * 16);
            }
        }
    }
    template <int BUF, bool FIRST>
    __device__ __forceinline__ void products(int half) {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < AH; ++i) {
                f32x4& d = dot[half * AH + i][j];
                d = Half<T>::mfma(b[j], fa[BUF][i], FIRST ? zero : d);
            }
    }
    __device__ __forceinline__ void finish_unit() {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float d = dot[i][j][e];
                    if constexpr (EACH) d = __builtin_fmaf(point[j][e], a_sum[i / 4][i % 4], d);
                    this->acc[i][j][e] = __builtin_fmaf(scale[j][e], d, this->acc[i][j][e]);
                }
        // (here: moved down to the slab's end, as they would be, a unit's products would take registers until then)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(this->acc[i][j]));
    }
    // acc += zeros * sums over units u0 .. end - 1, four of them a step, each eight k of the instruction: a float is cut into
    // three bf16 parts h, m, l that hold all its bits, and of the nine products all but l * l are taken.
    static __device__ __forceinline__ void cut(float v, uint32_t& h, uint32_t& m, uint32_t& l) {
        h = __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u;
        v -= __builtin_bit_cast(float, h);
        m = __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u;
        l = __builtin_bit_cast(uint32_t, v - __builtin_bit_cast(float, m));
    }
    static __device__ __forceinline__ uint32_t tops(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
    __device__ __forceinline__ void zero_points(const W4Tile& p, int tm, int tn, int u0, int end) {
        const int lane = lane_id(), r = lane % 16, g = lane / 16;
        const char* sums = p.sums + ((int64_t)tm * BM + r * TM) * 4;
        const char* zeros = p.zeros + ((int64_t)tn * kBN + wave_id() * 32 + r) * 4;
        const int64_t sum_step = (int64_t)p.g.tiles_m * BM * 4, zero_step = (int64_t)p.g.tiles_n * kBN * 4;
        f32x4 sum[TM / 4];
        float zero[TN];
        auto load = [&](int u) {   // (past the end: the last one's)
            const int at = min(u + g, end - 1);
#pragma unroll
            for (int i = 0; i < TM / 4; ++i) sum[i] = *reinterpret_cast<const f32x4*>(sums + at * sum_step + i * 16);
#pragma unroll
            for (int j = 0; j < TN; ++j) zero[j] = *reinterpret_cast<const float*>(zeros + at * zero_step + j * 64);
        };
        load(u0);
        for (int u = u0; u < end; u += 4) {
            uint32_t h, m, l;
            u32x4 zb[TN], sb[TM];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                cut(u + g < end ? zero[j] : 0.0f, h, m, l);
                zb[j] = u32x4{tops(h, m), tops(h, l), tops(m, h), tops(m, l)};
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                cut(u + g < end ? sum[i / 4][i % 4] : 0.0f, h, m, l);
                sb[i] = u32x4{tops(h, h), tops(m, h), tops(m, l), tops(l, m)};
            }
            load(u + 4);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) this->acc[i][j] = Half<DT_BF16>::mfma(zb[j], sb[i], this->acc[i][j]);
        }
    }
    template <int BUF>
    __device__ __forceinline__ void step(int q) {
        if (q % 2 == 0) {
#pragma unroll
            for (int j = 0; j < TN; ++j) b[j] = spread.in_order(word[j]);
        }
        if (S1) {
            products<BUF, true>(q % 2);
            if (q % 2 == 1) finish_unit();
        } else {
            if (q < 2 && pos == 0) products<BUF, true>(q % 2);
            else products<BUF, false>(q % 2);
            if (q == KS - 1) {
                --left;
                if (++pos == per_unit || left == 0) {
                    finish_unit();
                    pos = 0;
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void wait_lds() { wait_lgkm0(); }
    __device__ __forceinline__ void barrier() { gemm::barrier(); }
};

// Where chunk l (of UL) of what wave w copies lies for unit 0, in bytes from the sums, and the bytes from one unit to the next.
template <class F>
__device__ __forceinline__ uint32_t unit_chunk(const W4Tile& p, int tm, int tn, int w, int l) {
    if (l < 2 * F::SL)
        return (uint32_t)((l < F::SL ? p.scales : p.zeros) - p.sums) +
               (((uint32_t)(l % F::SL / 8) * p.g.tiles_n + tn) * kBN + w * (kBN / kNC)) * 4 + l % 8 * 16;
    l -= 2 * F::SL;
    return (((uint32_t)(l / F::RL) * p.g.tiles_m + tm) * (F::RL * 16) + (w * F::RL + l % F::RL) * 4) * 4;
}
template <class F>
__device__ __forceinline__ uint32_t unit_step(const W4Tile& p, int l) {
    return (uint32_t)(l < 2 * F::SL ? p.g.tiles_n * kBN : p.g.tiles_m * (F::RL * 16)) * 4;
}
// First unit of slab s of the whole K.
__device__ __forceinline__ int unit_of(const W4Tile& p, int s) { return p.per_unit ? s / p.per_unit : 2 * s; }

// Direct global -> LDS copies: 16-byte aligned rows, whole slabs and tiles.
template <int T, int BM, bool S1, bool EACH>
struct W4RingOps : W4Compute<T, BM, S1, EACH> {
    typedef W4Compute<T, BM, S1, EACH> F;
    ALoader<BM, 128, kNC> la;
    DirectLoader<kBN, 32, kNC, false> lq;
    static constexpr int ZL = EACH ? 2 * F::SL : F::SL;   // chunks of the scales, and of the zero points: one copy; the sums another
    static constexpr int L = decltype(la)::IPW + decltype(lq)::IPW + (EACH ? 2 : 1);
    const W4Tile* p;
    uint32_t at_scales, at_sums;
    int s0;
    __device__ __forceinline__ void init_units(const W4Tile& p_, int tm, int tn, int s0_) {
        p = &p_;
        s0 = s0_;
        at_scales = unit_chunk<F>(p_, tm, tn, wave_id(), lane_id());
        at_sums = EACH ? unit_chunk<F>(p_, tm, tn, wave_id(), ZL + lane_id()) : 0;
    }
    __device__ __forceinline__ void issue(int slab, int slot, int, int) {
        LDS_AS char* st = this->smem + slot * F::STAGE;
        la.issue(slab, st, 0, decltype(la)::IPW);
        lq.issue(slab, st + F::A_BYTES, 0, decltype(lq)::IPW);
        const int w = wave_id(), lane = lane_id(), u = unit_of(*p, s0 + slab);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)p->sums, (short)0, -1, kBufferFlags);
        if (lane < ZL) la.template copy<0>(rs, at_scales, u * unit_step<F>(*p, 0), st + F::S_AT + w * F::UL * 16);
        if constexpr (EACH) {
            if (lane < F::UL - ZL) la.template copy<0>(rs, at_sums, u * unit_step<F>(*p, ZL), st + F::S_AT + (w * F::UL + ZL) * 16);
        }
    }
    template <int N>
    __device__ __forceinline__ void wait_slabs() { wait_vm<N * L>(); }
    template <int BUF, int HAS, int PARTS>
    __device__ __forceinline__ void math(int q) { this->template step<BUF>(q); }
};

// Any pitch, alignment and size (K >= 64): 16-byte loads of any alignment into registers, one
// slab ahead, written into the other slot in the last step but one.  A chunk past a row's end is read
// as the row's last 16 bytes and shifted.  Rows past the end repeat the last.
template <int T, int BM, bool S1, bool EACH>
struct W4StagedOps : W4Compute<T, BM, S1, EACH> {
    typedef W4Compute<T, BM, S1, EACH> F;
    static constexpr int NT = 64 * kNC, STEP = NT / 8, CA = BM / STEP;
    static constexpr int UT = kNC * F::UL;   // threads with a chunk of the units
    static_assert(STEP % 16 == 0 && CA * STEP == BM && UT <= NT && 2 * kBN == NT, "chunks per thread");
    const char* arow[CA];
    const uint8_t* qrow;
    uint32_t uchunk, ustep;
    uint32_t dst;
    u32x4 va[CA], vq, vu;
    const W4Tile* p;
    int k_bytes, q_bytes, s0, wslot = 0, slab_ = 0;
    bool ask_write = false;
    __device__ __forceinline__ void init_rows(const W4Tile& p_, int tm, int tn, int m0, int n0, int s0_) {
        p = &p_;
        s0 = s0_;
        k_bytes = p->g.K * 2;
        q_bytes = (p->g.K + 1) / 2;
        const int t = threadIdx.x, row = t / 8, c = t % 8;
#pragma unroll
        for (int i = 0; i < CA; ++i) arow[i] = p->g.A + (int64_t)min(m0 + row + i * STEP, p->g.M - 1) * p->g.lda * 2;
        dst = (uint32_t)(row * 128 + ((c ^ swz<8>(row)) << 4));
        qrow = p->W + (int64_t)min(n0 + t / 2, p->g.N - 1) * p->ldw;
        uchunk = unit_chunk<F>(*p, tm, tn, t / F::UL % kNC, t % F::UL);
        ustep = unit_step<F>(*p, t % F::UL);
    }
    __device__ __forceinline__ void load(int slab) {
        slab_ = s0 + slab;
        const int ka = min(slab_ * 128 + (int)threadIdx.x % 8 * 16, k_bytes - 16);
        const int kq = min(slab_ * 32 + (int)threadIdx.x % 2 * 16, q_bytes - 16);
#pragma unroll
        for (int i = 0; i < CA; ++i) va[i] = load16(arow[i] + ka);
        vq = load16(qrow + kq);
        if ((int)threadIdx.x < UT) vu = load16(p->sums + (uchunk + (uint32_t)unit_of(*p, slab_) * ustep));
        ask_write = true;
    }
    __device__ __forceinline__ void put() {
        LDS_AS char* st = this->smem + wslot * F::STAGE;
        const int t = threadIdx.x;
        if ((slab_ + 1) * 128 > k_bytes) {   // the last slab, not filled
            const int by = slab_ * 128 + t % 8 * 16 + 16 - k_bytes;
#pragma unroll
            for (int i = 0; i < CA; ++i) va[i] = by > 0 ? shift_down(va[i], by) : va[i];
            const int byq = slab_ * 32 + t % 2 * 16 + 16 - q_bytes;
            vq = byq > 0 ? shift_down(vq, byq) : vq;
        }
#pragma unroll
        for (int i = 0; i < CA; ++i) *reinterpret_cast<LDS_AS u32x4*>(st + dst + i * STEP * 128) = va[i];
        *reinterpret_cast<LDS_AS u32x4*>(st + F::A_BYTES + (t ^ codes_swz(t / 2)) * 16) = vq;
        if (t < UT) *reinterpret_cast<LDS_AS u32x4*>(st + F::S_AT + t * 16) = vu;
        ask_write = false;
        wslot ^= 1;
    }
    __device__ __forceinline__ void write(int, int) {
        if (ask_write) put();   // (only slab 0 has not been written by math())
    }
    template <int BUF, int HAS, int PARTS>
    __device__ __forceinline__ void math(int q) {
        this->template step<BUF>(q);
        if (q == F::KS - 2 && ask_write) put();
    }
};

// Splits of K (blockIdx.y) store plain sums, each into its own buffer.
template <int T, int OUT, int BM, bool S1, bool EACH, bool DIRECT>
__global__ __launch_bounds__(64 * kNC) __attribute__((amdgpu_waves_per_eu(2)))
void w4_tile_kernel(W4Tile p) {
    typedef W4Compute<T, BM, S1, EACH> F;
    constexpr int S = DIRECT ? 3 : 2;
    __shared__ __attribute__((aligned(1024))) char smem_raw[S * F::STAGE];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    int tm, tn;
    tile_coords(p.g, tm, tn);
    const int m_keep = tm * BM, n_keep = tn * kBN;
    const int m0 = max(0, min(m_keep, p.g.M - BM)), n0 = max(0, min(n_keep, p.g.N - kBN));
    const int s0 = (int)blockIdx.y * p.per_split;
    const int slabs = min((p.g.K + kSlabK - 1) / kSlabK - s0, p.per_split);
    const int u0 = unit_of(p, s0), u1 = S1 ? u0 + 2 * slabs : u0 + (slabs + p.per_unit - 1) / p.per_unit;
    p.g.C += (int64_t)blockIdx.y * p.part;
    if constexpr (DIRECT) {
        W4RingOps<T, BM, S1, EACH> ops;
        ops.init(smem, p, slabs);
        ops.init_units(p, tm, tn, s0);
        init_a<BM, 128, kNC>(ops.la, p.g.A + ((int64_t)m0 * p.g.lda + (int64_t)s0 * kSlabK) * 2, p.g.lda * 2, kSlabK * 2, p.g.M - m0);
        ops.lq.init(reinterpret_cast<const char*>(p.W) + (int64_t)n0 * p.ldw + (int64_t)s0 * (kSlabK / 2), p.ldw, kSlabK / 2);
        const int lane = lane_id();
        ops.lq.vpat[0] = (uint32_t)(lane / 2 * (int)p.ldw + ((lane % 2) ^ codes_swz(lane / 2)) * 16);
        gemm_sched::ring_mainloop<S, F::KS, 1>(ops, slabs);
        if constexpr (!EACH) ops.zero_points(p, tm, tn, u0, u1);
        ops.template epilogue<OUT>(p.g, m0, n0, m_keep, n_keep);
    } else {
        W4StagedOps<T, BM, S1, EACH> ops;
        ops.init(smem, p, slabs);
        ops.init_rows(p, tm, tn, m0, n0, s0);
        gemm_sched::staged_mainloop<S, F::KS>(ops, slabs);
        if constexpr (!EACH) ops.zero_points(p, tm, tn, u0, u1);
        ops.template epilogue<OUT>(p.g, m0, n0, m_keep, n_keep);
    }
}

// Sums of A over units and the transposed scales.  Four lanes sum a unit of a row, 32 elements a turn; the
// workgroups behind those turn the scales; the first ones make the copies that the direct loads need, if any.
struct W4Prepare {
    const char* A;
    const uint16_t* scales;
    const uint16_t* zeros;
    float* sums;
    float* s;
    float* z;
    int64_t lda, lds;
    int M, N, K, group, unit, units, tiles_m, tiles_n, bm, tm;   // tm: blocks of 16 rows of a tile
    bool each;             // zero points by themselves, not times their scales
    int64_t sum_blocks;
    RowsJob pack_a, pack_w;
    uint32_t a_blocks, pack_blocks;
};
constexpr int kTurnCols = 64, kTurnUnits = 32;
template <int T>
__global__ __launch_bounds__(256) void w4_prepare_kernel(const W4Prepare p) {
    if (blockIdx.x < p.pack_blocks) {
        rows_pack(p.pack_a, p.pack_w, p.a_blocks, blockIdx.x);
        return;
    }
    const int64_t block = blockIdx.x - p.pack_blocks;
    if (block < p.sum_blocks) {
        const int64_t id = block * 64 + threadIdx.x / 4;   // (row of a tile, unit), the unit first
        const int64_t rows = (int64_t)p.tiles_m * p.bm;
        if (id >= rows * p.units) return;
        const int64_t row = id / p.units;
        const int u = (int)(id % p.units), tile = (int)(row / p.bm), local = (int)(row % p.bm);
        const int m = min(max(0, min(tile * p.bm, p.M - p.bm)) + local, p.M - 1);
        const char* a = p.A + (int64_t)m * p.lda * 2;
        float sum = 0.0f;
        const int end = (int)min((int64_t)(u + 1) * p.unit, (int64_t)p.K);
        for (int k = u * p.unit + (int)threadIdx.x % 4 * 8; k < end; k += 32) {
            const u32x4 v = load_a(a, k, p.K);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += to_f32<T>((uint16_t)v[e]) + to_f32<T>((uint16_t)(v[e] >> 16));
        }
        sum += __shfl_xor(sum, 1, 64);
        sum += __shfl_xor(sum, 2, 64);
        if (threadIdx.x % 4 == 0)
            p.sums[(int64_t)u * rows + (int64_t)tile * p.bm + local % 16 * p.tm + local / 16] = sum;   // a lane's tm sums side by side
        return;
    }
    // 64 columns by 32 units: read along the units of a column, written along the columns of a unit
    __shared__ uint32_t turn[kTurnUnits][kTurnCols + 1];
    const int64_t cols = (int64_t)p.tiles_n * kBN, id = block - p.sum_blocks;
    const int at0 = (int)(id % (cols / kTurnCols)) * kTurnCols, u0 = (int)(id / (cols / kTurnCols)) * kTurnUnits;
    const int ul = threadIdx.x % kTurnUnits;
#pragma unroll
    for (int c = threadIdx.x / kTurnUnits; c < kTurnCols; c += 256 / kTurnUnits) {
        const int at = at0 + c, n = min(max(0, min(at / kBN * kBN, p.N - kBN)) + at % kBN, p.N - 1);
        const int64_t k = (int64_t)(u0 + ul) * p.unit;
        uint32_t v = 0;   // a unit past the end: A is zero there
        if (k < p.K) {
            const int64_t i = n * p.lds + k / p.group;
            const uint16_t eight = T == DT_BF16 ? 0x4100 : 0x4800;
            v = p.scales[i] | (uint32_t)(p.zeros ? p.zeros[i] : eight) << 16;
        }
        turn[ul][c] = v;
    }
    __syncthreads();
#pragma unroll
    for (int u = threadIdx.x / kTurnCols; u < kTurnUnits; u += 256 / kTurnCols)
        if (u0 + u < p.units) {
            const int64_t i = (u0 + u) * cols + at0 + threadIdx.x % kTurnCols;
            const uint32_t v = turn[u][threadIdx.x % kTurnCols];
            const float s = to_f32<T>((uint16_t)v);
            p.s[i] = s;
            p.z[i] = (p.each ? -1.0f : -s) * zero16<T>((uint16_t)(v >> 16));
        }
}

// C = alpha * (sum of the splits, in order) + beta * C
template <int OUT>
__global__ __launch_bounds__(256) void w4_join_kernel(const GemmParams p, const char* part, int64_t each, int ldp, int splits) {
    const int64_t quads = ldp / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= quads * p.M) return;
    const int64_t m = id / quads;
    const int n = (int)(id % quads) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < splits; ++i) s += *reinterpret_cast<const f32x4*>(part + i * each + (m * ldp + n) * 4);
    store4<OUT>(p, m, n, s);
}

struct W4Plan {
    int bm, splits, unit, units, per_split;
    int64_t slabs, tiles_m, tiles_n;
    size_t sums, sz, parts;   // bytes of the workspace's pieces
    double us;                // what it is expected to take
};
// Measured times of the pieces, in microseconds: the launch that prepares, a workgroup's first loads and its stores, the
// launch that joins, a copy's bytes; and a slab, alone on its compute unit or with a second workgroup there, for
// units of 64 k or more and for short ones (tiles of 64 and 128 rows, 256 and 512 of them, K 1024 and 4096).
constexpr double kPrepareUs = 4.0, kFillUs = 3.0, kJoinUs = 5.0, kBytesPerUs = 4.5e6;
double slab_us(int bm, bool alone, bool short_units) {
    if (bm == 64) return alone ? (short_units ? 0.9 : 0.69) : (short_units ? 1.21 : 0.9);
    return alone ? (short_units ? 1.45 : 1.07) : (short_units ? 1.83 : 1.28);
}
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
int64_t ldp_of(int64_t N) { return (N + 3) / 4 * 4; }

// Tiles of 128 rows fill a compute unit with two workgroups of four waves (one of eight waves on 256 rows: 2048 x 14336 x 4096
// 313 us instead of 294: its group ends, barriers and stores have nothing to run under); tiles of 64 rows are for
// small problems.  Splits of K end with a unit; their sums are written and read once and take one more launch.
// Of both heights and all splits the one that should be fastest.
W4Plan w4_plan(int64_t M, int64_t N, int64_t K, int64_t group, size_t room) {
    W4Plan q = {};
    const int64_t cu = num_compute_units();
    q.tiles_n = ceil_div(N, kBN);
    q.slabs = ceil_div(K, kSlabK);
    q.unit = group % kSlabK == 0 ? (int)group : 32;
    q.units = (int)(q.unit == 32 ? 2 * q.slabs : ceil_div(K, group));
    q.sz = (size_t)q.units * q.tiles_n * kBN * 8;
    const int64_t per_unit = q.unit == 32 ? 1 : group / kSlabK, each = M * ldp_of(N) * 4;
    int64_t s = 1;
    for (int bm = 64; bm <= 128; bm += 64) {
        const int64_t tiles = ceil_div(M, bm) * q.tiles_n;
        const size_t sums = round256((size_t)q.units * ceil_div(M, bm) * bm * 4);
        for (int64_t t = 1; t <= 64 && t * 4 <= q.slabs + 3; ++t) {
            if (t > 1 && sums + q.sz + (size_t)(t * each) > room) break;
            const int64_t slabs = ceil_div(q.slabs, t), full = tiles * t / (2 * cu), rest = tiles * t % (2 * cu);
            double us = kPrepareUs + full * (kFillUs + slabs * slab_us(bm, false, q.unit == 32));
            if (rest) us += kFillUs + slabs * slab_us(bm, rest <= cu, q.unit == 32);
            if (t > 1) us += kJoinUs + t * each * 2.0 / kBytesPerUs;
            if (q.us == 0.0 || us < q.us) {
                q.us = us;
                q.bm = bm;
                q.sums = sums;
                s = t;
            }
        }
    }
    q.tiles_m = ceil_div(M, q.bm);
    q.per_split = (int)(ceil_div(ceil_div(q.slabs, s), per_unit) * per_unit);
    q.splits = (int)ceil_div(q.slabs, q.per_split);
    q.parts = q.splits > 1 ? (size_t)(q.splits * each) : 0;
    return q;
}

template <int T, int OUT, int BM, bool EACH>
hipError_t tile_of(const W4Tile& t, bool short_units, bool direct, int splits, hipStream_t st) {
    const dim3 grid((unsigned)(t.g.tiles_m * t.g.tiles_n), (unsigned)splits), block(256);
    if (short_units) {
        if (direct) hipLaunchKernelGGL((w4_tile_kernel<T, OUT, BM, true, EACH, true>), grid, block, 0, st, t);
        else hipLaunchKernelGGL((w4_tile_kernel<T, OUT, BM, true, EACH, false>), grid, block, 0, st, t);
    } else {
        if (direct) hipLaunchKernelGGL((w4_tile_kernel<T, OUT, BM, false, EACH, true>), grid, block, 0, st, t);
        else hipLaunchKernelGGL((w4_tile_kernel<T, OUT, BM, false, EACH, false>), grid, block, 0, st, t);
    }
    return hipGetLastError();
}
template <int T, int OUT, bool EACH>
hipError_t out_of(const W4Plan& q, const W4Tile& t, bool direct, hipStream_t st) {
    const bool s1 = q.unit == 32;
    if (q.bm == 128) return tile_of<T, OUT, 128, EACH>(t, s1, direct, q.splits, st);
    return tile_of<T, OUT, 64, EACH>(t, s1, direct, q.splits, st);
}

// What the direct loads need of A and the codes.  They hold a row's offset in its tile in 32 bits, as it lies in memory and
// as a copy lays it out: longer rows go through the staged loads, whose addresses are whole ones.
struct W4Copies {
    RowsJob a, w;
    bool copy_a, copy_w;   // whose rows they cannot read in place
    bool held;             // whether they can read the copies
    size_t bytes() const { return (copy_a ? a.bytes() : 0) + (copy_w ? w.bytes() : 0); }
};
W4Copies copies_of(const W4Params& f, const W4Plan& q) {
    const int64_t kp = q.slabs * kSlabK;
    auto held = [](int64_t rows, int64_t pitch) { return rows * pitch < (int64_t(1) << 31); };
    W4Copies c;
    c.a = {reinterpret_cast<const uint8_t*>(f.A), nullptr, f.lda * 2, f.M, (int64_t)f.K * 2, std::max((int64_t)f.M, least_rows(q.bm)), kp * 2};
    c.w = {f.W, nullptr, f.ldw, f.N, ((int64_t)f.K + 1) / 2, std::max((int64_t)f.N, (int64_t)kBN), kp / 2};
    c.copy_a = f.K != kp || f.M < least_rows(q.bm) || ((uintptr_t)f.A | c.a.ld) % 16 || !held(q.bm, c.a.ld);
    c.copy_w = f.K != kp || f.N < kBN || ((uintptr_t)f.W | c.w.ld) % 16 || !held(kBN, c.w.ld);
    c.held = (!c.copy_a || held(q.bm, c.a.len_pad)) && (!c.copy_w || held(kBN, c.w.len_pad)) &&
             c.bytes() < (size_t(1) << 34);   // (rows_pack counts chunks in 32 bits)
    return c;
}

template <int T>
hipError_t run_tiles(const W4Params& f, const W4Plan& q, char* ws, size_t ws_bytes, hipStream_t st) {
    W4Prepare a = {};
    a.A = f.A;
    a.scales = reinterpret_cast<const uint16_t*>(f.scales);
    a.zeros = reinterpret_cast<const uint16_t*>(f.zeros);
    a.sums = reinterpret_cast<float*>(ws);
    a.s = reinterpret_cast<float*>(ws + q.sums);
    a.z = reinterpret_cast<float*>(ws + q.sums + q.sz / 2);
    a.lda = f.lda; a.lds = f.lds;
    a.M = f.M; a.N = f.N; a.K = f.K; a.group = f.group;
    a.unit = q.unit; a.units = q.units;
    a.tiles_m = (int)q.tiles_m; a.tiles_n = (int)q.tiles_n;
    a.bm = q.bm; a.tm = q.bm / 16;
    const bool each = f.out_type == DT_F32;   // (see above: what a 16-bit C hides)
    a.each = each;
    a.sum_blocks = ceil_div(q.tiles_m * q.bm * q.units, 64);
    W4Tile t = {};
    GemmParams& p = t.g;
    p.A = f.A;
    p.C = f.C;
    p.lda = f.lda; p.ldc = f.ldc;
    p.M = f.M; p.N = f.N; p.K = f.K;
    p.alpha = 16.0f * f.alpha;   // the codes are sixteenths
    p.beta = f.beta;
    p.out_type = f.out_type;
    p.tiles_m = (int)q.tiles_m; p.tiles_n = (int)q.tiles_n;
    p.group_m = 8;
    p.xcd_remap = 1;
    // operands that the direct copies cannot take, copied behind the rest where there is room
    W4Copies c = copies_of(f, q);
    const size_t used = q.sums + q.sz + round256(q.parts);
    const bool copies = (c.copy_a || c.copy_w) && c.held && used + c.bytes() <= ws_bytes;
    const bool direct = copies || (!c.copy_a && !c.copy_w);
    op_note("  %d x %d tiles, units of %d, %d splits of K, %s loads%s", q.bm, kBN, q.unit, q.splits, direct ? "direct" : "staged",
            copies ? " of copied rows" : "");
    t.W = f.W;
    t.ldw = f.ldw;
    if (copies) {
        uint8_t* at = reinterpret_cast<uint8_t*>(ws) + used;
        if (c.copy_a) {
            c.a.dst = at;
            at += c.a.bytes();
            a.pack_a = c.a;
            a.a_blocks = a.pack_blocks = rows_pack_blocks(c.a);
            p.A = reinterpret_cast<const char*>(c.a.dst);
            p.lda = c.a.len_pad / 2;
        }
        if (c.copy_w) {
            c.w.dst = at;
            a.pack_w = c.w;
            a.pack_blocks += rows_pack_blocks(c.w);
            t.W = c.w.dst;
            t.ldw = c.w.len_pad;
        }
    }
    hipLaunchKernelGGL(w4_prepare_kernel<T>, dim3((unsigned)(a.pack_blocks + a.sum_blocks + q.tiles_n * (kBN / kTurnCols) * ceil_div(q.units, kTurnUnits))), dim3(256), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    t.sums = ws;
    t.scales = ws + q.sums;
    t.zeros = ws + q.sums + q.sz / 2;
    t.per_unit = q.unit == 32 ? 0 : q.unit / kSlabK;
    t.per_split = q.per_split;
    if (q.splits > 1) {
        const GemmParams whole = p;
        const int64_t ldp = ldp_of(f.N);
        char* parts = ws + q.sums + q.sz;
        t.part = f.M * ldp * 4;
        p.C = parts;
        p.ldc = ldp;
        p.alpha = 1.0f;
        p.beta = 0.0f;
        e = each ? out_of<T, DT_F32, true>(q, t, direct, st) : out_of<T, DT_F32, false>(q, t, direct, st);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)ceil_div(f.M * ldp / 4, 256));
        if (f.out_type == DT_F32) hipLaunchKernelGGL(w4_join_kernel<DT_F32>, grid, dim3(256), 0, st, whole, parts, t.part, (int)ldp, q.splits);
        else hipLaunchKernelGGL(w4_join_kernel<T>, grid, dim3(256), 0, st, whole, parts, t.part, (int)ldp, q.splits);
        return hipGetLastError();
    }
    return each ? out_of<T, DT_F32, true>(q, t, direct, st) : out_of<T, T, false>(q, t, direct, st);
}

}  // namespace

// Bytes for the sums, the scales, the splits and, for rows that whole slabs do not fill, the copies.
size_t w4_tile_workspace(int64_t M, int64_t N, int64_t K, int64_t group) {
    const W4Plan q = w4_plan(M, N, K, group, ~size_t(0) >> 1);
    W4Params f = {};
    f.M = (int)M; f.N = (int)N; f.K = (int)K;
    f.lda = K; f.ldw = (K + 1) / 2;   // (of contiguous operands)
    const W4Copies c = copies_of(f, q);
    return q.sums + q.sz + round256(q.parts) + (c.held ? c.bytes() : 0);
}

// Expected microseconds.
double w4_tile_us(const W4Params& f, size_t ws_bytes) {
    const W4Plan q = w4_plan(f.M, f.N, f.K, f.group, ws_bytes);
    const W4Copies c = copies_of(f, q);
    const double bytes = c.held ? (double)c.bytes() : 0.0;
    return q.us + (bytes > 0.0 ? 1.0 + 2.0 * bytes / kBytesPerUs : 0.0);
}

// K that the staged loads hold, grids and 32-bit offsets in range, and a workspace for the sums and scales.
bool w4_tile_fits(const W4Params& f, size_t ws_bytes) {
    if (f.K < kSlabK || f.K > (1 << 29)) return false;
    const W4Plan q = w4_plan(f.M, f.N, f.K, f.group, ws_bytes);
    return q.sums + q.sz + q.parts <= ws_bytes && q.tiles_m * q.tiles_n < (int64_t(1) << 22) &&
           (q.sums + q.sz) / 4 < (size_t(1) << 30);
}

hipError_t launch_w4_tile(int in_type, const W4Params& f, void* ws, size_t ws_bytes, hipStream_t st) {
    const W4Plan q = w4_plan(f.M, f.N, f.K, f.group, ws_bytes);
    return in_type == DT_BF16 ? run_tiles<DT_BF16>(f, q, static_cast<char*>(ws), ws_bytes, st)
                              : run_tiles<DT_F16>(f, q, static_cast<char*>(ws), ws_bytes, st);
}

}  // namespace gemm
