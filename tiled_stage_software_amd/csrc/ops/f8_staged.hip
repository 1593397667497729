// f8_staged.hip -- C = alpha * diag(sa) * (A * B^T) * diag(sb) + beta * C for e4m3 operands of
// any size, pitch and alignment: 64 x 64 tiles, four waves of 32 x 32, slabs of 128 bytes of K
// through registers into two LDS slots (staged_mainloop's protocol with one step a slab).
//
// The scales multiply the fp32 sum, so no operand is rounded again.
#include "f8_common.hpp"

namespace gemm {
namespace {

constexpr int kTile = 64, kSlab = 128, kStagedThreads = 256;
constexpr int kRows = 2 * kTile;                        // rows of A, then of B
constexpr int kSlot = kRows * kSlab;
constexpr int kPer = kRows * (kSlab / 16) / kStagedThreads;   // 16-byte chunks per thread and slab

template <bool WIDE>
__global__ __launch_bounds__(kStagedThreads) void f8_staged_kernel(const F8Params p, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[2 * kSlot];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    const int m0 = (int)(blockIdx.x / tiles_n) * kTile, n0 = (int)(blockIdx.x % tiles_n) * kTile;
    const int lane = lane_id(), w = wave_id();
    const int r = lane % 16, g = lane / 16;
    const int numK = (p.K + kSlab - 1) / kSlab;

    // thread t moves chunk t % 8 of rows t / 8, t / 8 + 32, ...; rows past the end repeat the last
    const uint8_t* src[kPer];
    uint32_t dst[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int row = (int)threadIdx.x / 8 + i * (kStagedThreads / 8), c = threadIdx.x % 8;
        src[i] = row < kTile ? p.A + (int64_t)min(m0 + row, p.M - 1) * p.lda
                             : p.B + (int64_t)min(n0 + row - kTile, p.N - 1) * p.ldb;
        dst[i] = (uint32_t)(row * kSlab + ((c ^ swz<8>(row)) << 4));
    }
    u32x4 v[kPer];
    auto load = [&](int kt) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = load_chunk(src[i], kt * kSlab + ((int)threadIdx.x % 8) * 16, p.K);
    };
    auto write = [&](int slot) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) *reinterpret_cast<LDS_AS u32x4*>(smem + slot * kSlot + dst[i]) = v[i];
    };

    const int wm = (w / 2) * 32, wn = (w % 2) * 32;
    // lane group g holds chunks kc and kc + 4 of the slab (0, 2, 1, 3: no bank conflicts)
    const int kc = (g & 1) * 2 + (g >> 1);
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto frag = [&](int slot, int row) {
        LDS_AS const char* s = smem + slot * kSlot + (row + r) * kSlab;
        const int sw = swz<8>(r);   // rows start at multiples of 16, the swizzle's period
        return join16(*reinterpret_cast<LDS_AS const u32x4*>(s + ((kc ^ sw) << 4)),
                      *reinterpret_cast<LDS_AS const u32x4*>(s + (((kc + 4) ^ sw) << 4)));
    };

    load(0);
    write(0);
    __syncthreads();
    for (int kt = 0; kt < numK; ++kt) {
        const int slot = kt & 1;
        if (kt + 1 < numK) load(kt + 1);
        i32x8 a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = frag(slot, wm + 16 * i);
            b[i] = frag(slot, kTile + wn + 16 * i);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma_f8<WIDE>(b[j], a[i], acc[i][j]);
        if (kt + 1 < numK) write(slot ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = m0 + wm + 16 * i + r;
        if (m >= p.M) continue;
        const float sa = scale_or_one(p.sa, m);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + wn + 16 * j + 4 * g + e;
                if (n < p.N)
                    store_c1(p.C, p.out_type, (int64_t)m * p.ldc + n, acc[i][j][e] * sa * scale_or_one(p.sb, n),
                             p.alpha, p.beta);
            }
    }
}

}  // namespace

hipError_t launch_f8_staged(const F8Params& f, hipStream_t st) {
    const int64_t cols = f.N < kMostCols ? f.N : kMostCols, most = INT32_MAX / kStagedThreads;   // tiles of a launch
    return in_pieces(f, most / ((cols + kTile - 1) / kTile) * kTile, cols, [&](const F8Params& p) {
        const int64_t tm = ((int64_t)p.M + kTile - 1) / kTile, tn = ((int64_t)p.N + kTile - 1) / kTile;
        const dim3 grid((unsigned)(tm * tn)), block(kStagedThreads);
        if (p.out_type == DT_F32) hipLaunchKernelGGL(f8_staged_kernel<true>, grid, block, 0, st, p, (int)tn);
        else hipLaunchKernelGGL(f8_staged_kernel<false>, grid, block, 0, st, p, (int)tn);
        return hipGetLastError();
    });
}

}  // namespace gemm
