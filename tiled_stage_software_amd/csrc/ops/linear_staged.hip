// linear_staged.hip -- the product with bias, activation and residual for operands of any size, pitch and
// alignment: 128 x 128 tiles, slabs of 64 in two LDS slots, loads through registers, zeros past the edges (no K at all
// leaves act(bias) + R).  For what the other kernels do not take: K below 64 and pitches above 2^21.  K below 64 takes three times its
// bytes (4096 x 4096 x 32 bf16 21.8 us, floor 6.6; 8192 x 14336 x 32 124, floor 46; the same from K = 8 to 48): a workgroup's loads, products
// and epilogue run in turn, and LDS holds two of them a compute unit.
#include "linear.hpp"

namespace gemm {
namespace {

constexpr int kBM = 128, kBN = 128, kBK = 64;

template <int T, int OUT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void linear_staged_kernel(const GemmParams p, const LinearEpi e) {
    typedef MfmaStagedOps<half_of<T>, kBM, kBN, kBK, 2, 2, 2, false, false> Ops;
    __shared__ __attribute__((aligned(1024))) char smem_raw[2 * Ops::STAGE];
    LDS_AS char* smem = (LDS_AS char*)smem_raw;
    int tm, tn;
    tile_coords(p, tm, tn);
    const int m0 = tm * kBM, n0 = tn * kBN;
    Ops ops;
    ops.init(smem);
    ops.la.init(p.A, p.lda, m0, 0, p.M, p.K, p.a_vec != 0, false);
    ops.lb.init(p.B, p.ldb, n0, 0, p.N, p.K, p.b_vec != 0, false);
    gemm_sched::staged_mainloop<2, Ops::KS>(ops, (p.K + kBK - 1) / kBK);
    linear_epilogue<T, OUT, kBM, kBN, 2, 2, 32, 2 * Ops::STAGE>(ops, e, smem, m0, n0, m0, n0);
}

}  // namespace

hipError_t launch_linear_staged(int in_type, const LinearParams& f, hipStream_t st) {
    return in_pieces(f, int64_t(1) << 18, int64_t(1) << 18, [&](const LinearParams& q) {
        GemmParams p = {};
        p.A = q.A;
        p.B = q.W;
        p.lda = q.lda; p.ldb = q.ldw;
        p.M = q.M; p.N = q.N; p.K = q.K;
        p.tiles_m = (q.M + kBM - 1) / kBM;
        p.tiles_n = (q.N + kBN - 1) / kBN;
        p.group_m = 8;
        p.xcd_remap = 1;
        p.a_vec = ((uintptr_t)q.A | (uint64_t)q.lda * 2) % 16 == 0;
        p.b_vec = ((uintptr_t)q.W | (uint64_t)q.ldw * 2) % 16 == 0;
        return by_type(in_type, q.out_type, [&](auto t, auto o) {
            hipLaunchKernelGGL((linear_staged_kernel<decltype(t)::value, decltype(o)::value>), dim3((unsigned)(p.tiles_m * p.tiles_n)),
                               dim3(256), 0, st, p, epi_of(q));
            return hipGetLastError();
        });
    });
}

}  // namespace gemm
