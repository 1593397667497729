// short_loader.hpp -- direct global -> LDS copies of a small tile's rows that may be fewer than the tile's.
//
// As DirectLoader, but each copy has its own lane offsets instead of one scalar row offset, in which rows past the
// end repeat the last: a tile of 64 rows has two copies a wave, so that is two registers and one more write of M0 a slab.
// Without it an operand of 33 to 63 rows is first copied to whole tiles (8 bits, 33 x 14336 x 4096: 16.4 us instead of 13.1).
#pragma once

#include <type_traits>

#include "../mfma.hpp"

namespace gemm {

template <int LR, int ROWB, int NW>
struct ShortLoader : DirectLoader<LR, ROWB, NW, true> {
    typedef DirectLoader<LR, ROWB, NW, true> D;
    uint32_t at[D::IPW];   // per lane: its row's and chunk's offset in copy i
    // rows: those that there are, LR or fewer; the host keeps rows * ld_bytes < 2^31.
    __device__ __forceinline__ void init(const char* row_origin, int64_t ld_bytes, int64_t slab_bytes, int rows) {
        const int w = wave_id(), lane = lane_id();
        this->base = row_origin;
        this->slab_step = slab_bytes;
        this->lds_wave = w * D::IPW * 1024;
#pragma unroll
        for (int i = 0; i < D::IPW; ++i) {
            const int row = (w * D::IPW + i) * D::RPI + lane / D::CPR;
            const int c = lane % D::CPR ^ swz<D::CPR>(row);
            at[i] = (uint32_t)min(row, rows - 1) * (uint32_t)ld_bytes + c * 16;
        }
    }
    __device__ __forceinline__ void issue(int slab, LDS_AS char* lds_tile, int i0, int i1) const {
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void*)(this->base + (int64_t)slab * this->slab_step), (short)0, -1, kBufferFlags);
#pragma unroll
        for (int i = 0; i < D::IPW; ++i)
            if (i >= i0 && i < i1) D::template copy<0>(rs, at[i], 0, lds_tile + this->lds_wave + i * 1024);
    }
};

// The loader of A's rows in tiles of BM rows.
constexpr int kShortRows = 64;
// Rows of A that direct copies into tiles of bm rows need.
constexpr int64_t least_rows(int bm) { return bm == kShortRows ? 1 : bm; }
template <int BM, int ROWB, int NW>
using ALoader = std::conditional_t<BM == kShortRows, ShortLoader<BM, ROWB, NW>, DirectLoader<BM, ROWB, NW, true>>;
template <int BM, int ROWB, int NW>
__device__ __forceinline__ void init_a(ALoader<BM, ROWB, NW>& la, const char* row_origin, int64_t ld_bytes, int64_t slab_bytes, int rows) {
    if constexpr (BM == kShortRows) la.init(row_origin, ld_bytes, slab_bytes, min(rows, BM));
    else la.init(row_origin, ld_bytes, slab_bytes);
}

}  // namespace gemm
