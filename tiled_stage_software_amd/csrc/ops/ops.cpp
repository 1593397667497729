// ops.cpp -- the C entry points of the operators around the products: argument checks,
// kernel choice and launch.  Checks run before anything is enqueued.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "ops.hpp"

namespace {

using namespace gemm;

constexpr int64_t kMaxSize = int64_t(1) << 30;
constexpr int64_t kWsAlign = 256;

#define REQUIRE(cond, ...)                                                   \
    do {                                                                     \
        if (!(cond)) return op_fail(GEMM_ERR_INVALID_ARG, __VA_ARGS__);      \
    } while (0)

bool float_type(int t) { return t == GEMM_F32 || t == GEMM_BF16 || t == GEMM_F16; }

gemm_status_t check_size(const char* what, int64_t v) {
    REQUIRE(v >= 0 && v <= kMaxSize, "%s=%lld: sizes are 0..2^30", what, (long long)v);
    return GEMM_OK;
}
gemm_status_t check_ld(const char* what, int64_t ld, int64_t least) {
    REQUIRE(ld >= 1 && ld >= least, "%s=%lld < %lld", what, (long long)ld, (long long)least);
    return GEMM_OK;
}
gemm_status_t check_ws(const void* ws) {
    REQUIRE(reinterpret_cast<uintptr_t>(ws) % kWsAlign == 0, "workspace must be %lld-byte aligned", (long long)kWsAlign);
    return GEMM_OK;
}
#define TRY(expr)                              \
    do {                                       \
        const gemm_status_t s_ = (expr);       \
        if (s_ != GEMM_OK) return s_;          \
    } while (0)

gemm_status_t launched(hipError_t e) {
    if (e != hipSuccess) return op_fail(GEMM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return GEMM_OK;
}

gemm_status_t check_product(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldc, const void* C, const void* ws) {
    TRY(check_size("M", M));
    TRY(check_size("N", N));
    TRY(check_size("K", K));
    TRY(check_ld("lda", lda, K));
    TRY(check_ld("ldc", ldc, N));
    TRY(check_ws(ws));
    REQUIRE(M == 0 || N == 0 || C, "C is NULL");
    return GEMM_OK;
}

// C = beta * C, what is left of a product with K == 0 or alpha == 0.
gemm_status_t scale_only(int64_t M, int64_t N, float beta, void* C, int c_type, int64_t ldc, hipStream_t st) {
    GemmParams p;
    memset(&p, 0, sizeof(p));
    p.C = static_cast<char*>(C);
    p.ldc = ldc;
    p.M = (int)M;
    p.N = (int)N;
    p.beta = beta;
    p.out_type = c_type;
    return launched(launch_scale(p, st));
}

// Parts the rows of the backward pass are cut into with this much workspace.
int parts_for(int in_type, int64_t rows, int64_t cols, size_t bytes) {
    const int want = norm_bwd_parts(in_type, rows, (int)cols);
    const int64_t fit = (int64_t)(bytes / ((size_t)cols * sizeof(float)));
    return fit < 2 ? 1 : fit < want ? (int)fit : want;
}

// Whether the kernel for few rows takes a product: tiles of 64 rows read B with fewer, larger copies, which wins where many
// rows of B meet 17 rows of A or more, or a short K (17 x 14336 x 4096: 18 us instead of 22; 16 x 28672 x 1024: 7.5 instead of
// 15.8).  Only where it should win clearly: up to 16 rows both read B as fast as the card lets them when K is long.
bool f8_few(const F8Params& p, size_t ws_bytes) {
    if (p.M > kF8SkinnyRows) return false;
    return !f8_tile_fits(p) || f8_tile_us(p, ws_bytes) > (p.M > 16 ? 0.85 : 0.7) * f8_skinny_us(p);
}

}  // namespace

extern "C" {

gemm_status_t gemm_rmsnorm(gemm_dtype_t in_type, gemm_dtype_t w_type, gemm_dtype_t y_type, int64_t rows, int64_t cols,
                           float eps, const void* x, int64_t ldx, const void* r, int64_t ldr, const void* w, void* h,
                           int64_t ldh, void* y, int64_t ldy, float* scale, float* rstd, hipStream_t stream) {
    op_clear_error();
    REQUIRE(float_type(in_type), "in_type %d", (int)in_type);
    REQUIRE(!w || w_type == in_type || w_type == GEMM_F32, "w_type %d not offered for in_type %d", (int)w_type, (int)in_type);
    REQUIRE(float_type(y_type) || y_type == GEMM_F8E4M3, "y_type %d", (int)y_type);
    TRY(check_size("rows", rows));
    TRY(check_size("cols", cols));
    REQUIRE(eps >= 0.0f && isfinite(eps), "eps=%g", (double)eps);
    TRY(check_ld("ldx", ldx, cols));
    if (r) TRY(check_ld("ldr", ldr, cols));
    if (h) TRY(check_ld("ldh", ldh, cols));
    TRY(check_ld("ldy", ldy, cols));
    if (rows == 0 || cols == 0) return GEMM_OK;
    REQUIRE(x, "x is NULL");
    REQUIRE(y, "y is NULL");
    REQUIRE(scale || y_type != GEMM_F8E4M3, "scale is NULL");
    NormParams p;
    p.x = static_cast<const char*>(x);
    p.r = static_cast<const char*>(r);
    p.w = static_cast<const char*>(w);
    p.h = static_cast<char*>(h);
    p.y = static_cast<char*>(y);
    p.scale = scale;
    p.rstd = rstd;
    p.ldx = ldx; p.ldr = r ? ldr : 0; p.ldh = h ? ldh : 0; p.ldy = ldy;
    p.rows = rows;
    p.cols = (int)cols;
    p.w_type = w_type;
    p.y_type = y_type;
    p.eps = eps;
    op_note("rmsnorm type %d -> %d rows=%lld cols=%lld residual=%d weights=%d", (int)in_type, (int)y_type, (long long)rows,
            (long long)cols, r != nullptr, w ? (int)w_type : -1);
    return launched(launch_norm(in_type, p, stream));
}

gemm_status_t gemm_rmsnorm_bwd(gemm_dtype_t in_type, gemm_dtype_t w_type, int64_t rows, int64_t cols, const void* dy,
                               int64_t lddy, const void* h, int64_t ldh, const void* w, const float* rstd,
                               const void* dh, int64_t lddh, void* dx, int64_t lddx, float* dw, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    op_clear_error();
    REQUIRE(float_type(in_type), "in_type %d", (int)in_type);
    REQUIRE(!w || w_type == in_type || w_type == GEMM_F32, "w_type %d not offered for in_type %d", (int)w_type, (int)in_type);
    TRY(check_size("rows", rows));
    TRY(check_size("cols", cols));
    TRY(check_ld("lddy", lddy, cols));
    TRY(check_ld("ldh", ldh, cols));
    if (dh) TRY(check_ld("lddh", lddh, cols));
    TRY(check_ld("lddx", lddx, cols));
    TRY(check_ws(workspace));
    if (cols == 0 || (rows == 0 && !dw)) return GEMM_OK;
    if (rows > 0) {
        REQUIRE(dy, "dy is NULL");
        REQUIRE(h, "h is NULL");
        REQUIRE(rstd, "rstd is NULL");
        REQUIRE(dx, "dx is NULL");
    }
    NormBwdParams p;
    p.dy = static_cast<const char*>(dy);
    p.h = static_cast<const char*>(h);
    p.w = static_cast<const char*>(w);
    p.rstd = rstd;
    p.dh = static_cast<const char*>(dh);
    p.dx = static_cast<char*>(dx);
    p.dw = dw;
    p.part = static_cast<float*>(workspace);
    p.lddy = lddy; p.ldh = ldh; p.lddh = dh ? lddh : 0; p.lddx = lddx;
    p.rows = rows;
    p.cols = (int)cols;
    p.w_type = w_type;
    // (without dw there are no partial sums to keep)
    p.parts = dw ? parts_for(in_type, rows, cols, workspace ? workspace_bytes : 0) : norm_bwd_parts(in_type, rows, (int)cols);
    op_note("rmsnorm_bwd type %d rows=%lld cols=%lld in %d parts", (int)in_type, (long long)rows, (long long)cols, p.parts);
    return launched(launch_norm_bwd(in_type, p, stream));
}

gemm_status_t gemm_rmsnorm_bwd_workspace_size(gemm_dtype_t in_type, int64_t rows, int64_t cols, size_t* bytes) {
    op_clear_error();
    REQUIRE(bytes, "bytes is NULL");
    *bytes = 0;
    REQUIRE(float_type(in_type), "in_type %d", (int)in_type);
    TRY(check_size("rows", rows));
    TRY(check_size("cols", cols));
    const int parts = cols > 0 ? norm_bwd_parts(in_type, rows, (int)cols) : 0;
    if (parts > 1) *bytes = (size_t)parts * (size_t)cols * sizeof(float);
    return GEMM_OK;
}

gemm_status_t gemm_f8(int64_t M, int64_t N, int64_t K, float alpha, const void* A, int64_t lda, const float* scale_a,
                      const void* B, int64_t ldb, const float* scale_b, float beta, void* C, gemm_dtype_t c_type,
                      int64_t ldc, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    op_clear_error();
    REQUIRE(float_type(c_type), "c_type %d", (int)c_type);
    TRY(check_product(M, N, K, lda, ldc, C, workspace));
    TRY(check_ld("ldb", ldb, K));
    if (M == 0 || N == 0) return GEMM_OK;
    if (K == 0 || alpha == 0.0f) return scale_only(M, N, beta, C, c_type, ldc, stream);
    REQUIRE(A, "A is NULL");
    REQUIRE(B, "B is NULL");
    F8Params p;
    p.A = static_cast<const uint8_t*>(A);
    p.B = static_cast<const uint8_t*>(B);
    p.C = static_cast<char*>(C);
    p.sa = scale_a;
    p.sb = scale_b;
    p.lda = lda; p.ldb = ldb; p.ldc = ldc;
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.alpha = alpha; p.beta = beta;
    p.out_type = c_type;
    if (!workspace) workspace_bytes = 0;
    const bool few = f8_few(p, workspace_bytes), tiles = !few && f8_tile_fits(p);
    op_note("f8 -> type %d M=%lld N=%lld K=%lld: %s", (int)c_type, (long long)M, (long long)N, (long long)K,
            few ? "few rows" : tiles ? "tiles" : "64 x 64 tiles");
    if (few) return launched(launch_f8_skinny(p, stream));
    return launched(tiles ? launch_f8_tile(p, workspace, workspace_bytes, stream) : launch_f8_staged(p, stream));
}

gemm_status_t gemm_f8_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
    op_clear_error();
    REQUIRE(bytes, "bytes is NULL");
    *bytes = 0;
    TRY(check_size("M", M));
    TRY(check_size("N", N));
    TRY(check_size("K", K));
    if (M > 0 && N > 0 && K > 0)
        for (const gemm_dtype_t c_type : {GEMM_BF16, GEMM_F32}) {   // (the type of C is not known here: the larger of the two)
            F8Params p = {};
            p.M = (int)M; p.N = (int)N; p.K = (int)K;
            p.lda = p.ldb = K;   // (of contiguous operands)
            p.out_type = c_type;
            if (!f8_tile_fits(p) || f8_few(p, SIZE_MAX / 2)) continue;   // (the other kernels use none)
            *bytes = std::max(*bytes, f8_tile_workspace(p));
        }
    return GEMM_OK;
}

gemm_status_t gemm_w4(gemm_dtype_t in_type, int64_t M, int64_t N, int64_t K, int64_t group, float alpha, const void* A,
                      int64_t lda, const void* codes, int64_t ldw, const void* scales, const void* zeros, int64_t lds,
                      float beta, void* C, gemm_dtype_t c_type, int64_t ldc, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    op_clear_error();
    REQUIRE(in_type == GEMM_BF16 || in_type == GEMM_F16, "in_type %d: A is bf16 or f16", (int)in_type);
    REQUIRE(c_type == GEMM_F32 || c_type == in_type, "c_type %d not offered for in_type %d", (int)c_type, (int)in_type);
    TRY(check_product(M, N, K, lda, ldc, C, workspace));
    REQUIRE(group >= 32 && group % 32 == 0 && group <= kMaxSize, "group=%lld: a multiple of 32", (long long)group);
    TRY(check_ld("ldw", ldw, (K + 1) / 2));
    TRY(check_ld("lds", lds, (K + group - 1) / group));
    if (M == 0 || N == 0) return GEMM_OK;
    if (K == 0 || alpha == 0.0f) return scale_only(M, N, beta, C, c_type, ldc, stream);
    REQUIRE(A, "A is NULL");
    REQUIRE(codes, "codes is NULL");
    REQUIRE(scales, "scales is NULL");
    W4Params p;
    p.A = static_cast<const char*>(A);
    p.W = static_cast<const uint8_t*>(codes);
    p.scales = static_cast<const char*>(scales);
    p.zeros = static_cast<const char*>(zeros);
    p.C = static_cast<char*>(C);
    p.lda = lda; p.ldw = ldw; p.lds = lds; p.ldc = ldc;
    p.M = (int)M; p.N = (int)N; p.K = (int)K; p.group = (int)group;
    p.alpha = alpha; p.beta = beta;
    p.out_type = c_type;
    if (!workspace) workspace_bytes = 0;
    const bool vector = M <= kW4VectorRows;
    const bool tiles = !vector && w4_tile_fits(p, workspace_bytes) && w4_tile_us(p, workspace_bytes) < w4_skinny_us(p);
    op_note("w4 type %d -> %d M=%lld N=%lld K=%lld group=%lld: %s", (int)in_type, (int)c_type, (long long)M, (long long)N,
            (long long)K, (long long)group, vector ? "dot products" : tiles ? "tiles" : "few rows");
    if (vector) return launched(launch_w4_vector(in_type, p, stream));
    if (tiles) return launched(launch_w4_tile(in_type, p, workspace, workspace_bytes, stream));
    return launched(launch_w4_skinny(in_type, p, stream));
}

gemm_status_t gemm_w4_workspace_size(gemm_dtype_t in_type, int64_t M, int64_t N, int64_t K, int64_t group, size_t* bytes) {
    op_clear_error();
    REQUIRE(bytes, "bytes is NULL");
    *bytes = 0;
    REQUIRE(in_type == GEMM_BF16 || in_type == GEMM_F16, "in_type %d: A is bf16 or f16", (int)in_type);
    TRY(check_size("M", M));
    TRY(check_size("N", N));
    TRY(check_size("K", K));
    REQUIRE(group >= 32 && group % 32 == 0 && group <= kMaxSize, "group=%lld: a multiple of 32", (long long)group);
    if (M > kW4VectorRows && N > 0 && K > 0) {
        W4Params p = {};
        p.M = (int)M; p.N = (int)N; p.K = (int)K; p.group = (int)group;
        p.lda = K; p.ldw = (K + 1) / 2;   // (of contiguous operands)
        if (w4_tile_fits(p, SIZE_MAX / 2) && w4_tile_us(p, SIZE_MAX / 2) < w4_skinny_us(p)) *bytes = w4_tile_workspace(M, N, K, group);
    }
    return GEMM_OK;
}

}  // extern "C"
