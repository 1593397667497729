// block.cpp -- the C entry points of a transformer block's dense parts: the product with bias, activation and
// residual, the norm and rotation of heads, and their backward passes.  Checks run before anything is enqueued.
#include <math.h>

#include <algorithm>

#include "checks.hpp"

namespace {

using namespace gemm;

bool half_type(int t) { return t == GEMM_BF16 || t == GEMM_F16; }
int64_t round256(int64_t v) { return (v + 255) & ~int64_t(255); }

gemm_status_t check_linear(int in_type, int act, int64_t M, int64_t N, int64_t K) {
    REQUIRE(half_type(in_type), "in_type %d: bf16 or f16", in_type);
    REQUIRE(act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU, "act %d", act);
    TRY(check_size("M", M));
    TRY(check_size("N", N));
    TRY(check_size("K", K));
    return GEMM_OK;
}

// Whether the kernel for few rows takes a product.  Its workgroups' waves are bound by the steps of K that a compute unit has to take, and
// more so from rows that do not start at cache lines, where tiles have splits of K and fewer bytes of A to load.  Measured
// (bf16, microseconds, few rows / tiles): 32 rows 4096 x 4096 (64 steps) 10.5 / 12.6, 1152 x 12608 (197) 19.3 / 13.7, 4096 x 14336
// (224) 31.9 / 27.2, 14336 x 4096 (224) 39 / 27, 32768 x 2048 (256) 49 / 29; 16 rows 14336 x 4096 about even, 352 x 16000 (250) 15.0 /
// 11.4, rows 16 bytes further apart 35.8 / 28.9 and 20.1 / 12.7; one row 8044 x 15920 (490) 49 / 51.  Without the workspace that tiles ask for, always.
bool linear_few(const LinearParams& p, bool lines, size_t ws_bytes) {   // lines: W's rows start at cache lines
    if (p.M > kLinearSkinnyRows || p.K < 1) return false;
    const double steps = std::max(1.0, p.N / 16.0 / num_compute_units()) * p.K / 64.0;
    if (p.M <= 4 || steps <= (p.M <= 16 && lines ? 224.0 : 128.0) || !linear_tile_fits(p)) return true;
    LinearParams q = p;
    q.lda = q.ldw = p.K;
    return ws_bytes < linear_tile_workspace(q);
}

// One of the backward pass's products (rows_a: A is K x M in memory), where the tiles do not take it: through the library's own
// 16-bit entry points.
gemm_status_t product(int in_type, const GradParams& p, void* ws, size_t bytes, hipStream_t st) {
    return (in_type == GEMM_BF16 ? gemm_bf16_ws : gemm_f16_ws)(p.rows_a ? GEMM_COL_MAJOR : GEMM_ROW_MAJOR, GEMM_ROW_MAJOR, p.M, p.N, p.K, 1.0f,
                                                               p.A, p.lda, p.B, p.ldb, 0.0f, p.C, (gemm_dtype_t)p.out_type, p.ldc, st, nullptr,
                                                               bytes ? ws : nullptr, bytes);
}

bool aligned_rows(const void* at, int64_t ld, int64_t len) { return (uintptr_t)at % 16 == 0 && ld % 8 == 0 && len % 8 == 0; }
RowsJob rows_job(const void* src, int64_t ld, int64_t rows, int64_t len) {
    return RowsJob{static_cast<const uint8_t*>(src), nullptr, ld * 2, rows, len * 2, rows, (len + 7) / 8 * 16};
}

// What a backward pass makes of its workspace: partial sums of db; aligned copies of dZ, A and W; the products' splits.
struct BackwardPlan {
    GradParams f[2];     // dA, dW
    RowsJob copies[3];   // of dZ, A, W; no source: none
    int parts;           // of db
    size_t sums, bytes;  // db's, all
    bool tiles;          // the products run on tiles; else one after the other through the 16-bit entry points
};
BackwardPlan backward_plan(int64_t M, int64_t N, int64_t K, const void* dz, int64_t lddz, const void* A, int64_t lda, const void* W, int64_t ldw,
                           void* dA, int64_t ldda, int in_type, void* dW, int64_t lddw, int dw_type, bool db, size_t ws) {
    BackwardPlan b = {};
    auto text = [](const void* p) { return static_cast<const char*>(p); };
    b.f[0] = GradParams{text(dz), text(W), static_cast<char*>(dA), lddz, ldw, ldda, (int)M, (int)K, (int)N, false, in_type, 0, 0, 0, 1};
    b.f[1] = GradParams{text(dz), text(A), static_cast<char*>(dW), lddz, lda, lddw, (int)N, (int)K, (int)M, true, dw_type, 0, 0, 0, 1};
    b.parts = linear_bwd_parts(M, N);
    if (db) {   // (partial sums are needed for db alone)
        b.parts = (int)std::max<int64_t>(1, std::min<int64_t>(b.parts, (int64_t)(ws / ((size_t)std::max<int64_t>(N, 1) * sizeof(float)))));
        if (b.parts > 1) b.sums = std::min(ws, (size_t)round256((int64_t)b.parts * N * (int64_t)sizeof(float)));
    }
    b.bytes = b.sums;
    if (M == 0 || N == 0 || K == 0 || (!dA && !dW)) return b;
    // tiles take aligned rows: copies of the others, where there is room for them
    const bool copy[3] = {!aligned_rows(dz, lddz, N), dW && !aligned_rows(A, lda, K), dA && !aligned_rows(W, ldw, K)};
    const RowsJob jobs[3] = {rows_job(dz, lddz, M, N), rows_job(A, lda, M, K), rows_job(W, ldw, N, K)};
    size_t at = b.sums, of_copies = 0;
    b.tiles = true;
    for (int i = 0; i < 3; ++i)
        if (copy[i]) of_copies += (size_t)round256(jobs[i].bytes());
    if (at + of_copies > ws || of_copies >= (size_t(1) << 34)) b.tiles = of_copies == 0;
    GradParams aligned[2] = {b.f[0], b.f[1]};
    if (copy[0]) aligned[0].lda = aligned[1].lda = jobs[0].len_pad / 2;
    if (copy[1]) aligned[1].ldb = jobs[1].len_pad / 2;
    if (copy[2]) aligned[0].ldb = jobs[2].len_pad / 2;
    for (const GradParams& p : aligned)
        if (p.C && !linear_grad_fits(p)) b.tiles = false;
    if (!b.tiles) return b;
    for (int i = 0; i < 3; ++i)
        if (copy[i]) {
            b.copies[i] = jobs[i];
            at += (size_t)round256(jobs[i].bytes());
        }
    b.f[0] = aligned[0];
    b.f[1] = aligned[1];
    linear_grad_plan(b.f, ws - at);
    b.bytes = at + b.f[0].ws + b.f[1].ws;
    return b;
}

gemm_status_t check_heads(const char* what, const gemm_heads_t* h, int64_t tokens, int64_t heads, int64_t dim, HeadsTensor* to) {
    *to = HeadsTensor{nullptr, 0, 0};
    if (tokens == 0 || heads == 0) return GEMM_OK;
    REQUIRE(h && h->data, "%s is NULL", what);
    const int64_t ld = h->token_stride, hs = h->head_stride, most = int64_t(1) << 40;
    const bool one_token = tokens == 1, one_head = heads == 1;
    // from the first token (head) to the last: strides below 2^40 times up to 2^30 tokens do not fit 64 bits
    const __int128 token_span = one_token ? 0 : (__int128)(tokens - 1) * ld, head_span = one_head ? 0 : (__int128)(heads - 1) * hs;
    // tokens outermost or heads outermost: nothing of one lies within another
    const bool fine = (one_token || (ld > 0 && ld < most)) && (one_head || (hs > 0 && hs < most)) &&
                      ((one_head || hs >= dim) && (one_token || ld >= head_span + dim) || (one_token || ld >= dim) && (one_head || hs >= token_span + dim));
    REQUIRE(fine, "%s: heads overlap (token stride %lld, head stride %lld)", what, (long long)ld, (long long)hs);
    REQUIRE(token_span + head_span < (int64_t(1) << 60), "%s: offsets past 64 bits (token stride %lld, head stride %lld)", what, (long long)ld,
            (long long)hs);
    *to = HeadsTensor{static_cast<const char*>(h->data), one_token ? 0 : ld, one_head ? 0 : hs};
    return GEMM_OK;
}

// What both passes check, but for the tensors that they read and write.
gemm_status_t check_qk(int in_type, int w_type, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim, float eps,
                       const void* wq, const void* wk, const gemm_rope_t* rope, HeadsParams* p) {
    *p = HeadsParams{};
    REQUIRE(float_type(in_type), "in_type %d", in_type);
    REQUIRE((!wq && !wk) || w_type == in_type || w_type == GEMM_F32, "w_type %d not offered for in_type %d", w_type, in_type);
    TRY(check_size("tokens", tokens));
    REQUIRE(q_heads >= 0 && q_heads <= 65536, "q_heads=%lld: 0..65536", (long long)q_heads);
    REQUIRE(k_heads >= 0 && k_heads <= 65536, "k_heads=%lld: 0..65536", (long long)k_heads);
    REQUIRE(dim >= 1 && dim <= kMostHeadDim, "head_dim=%lld: 1..%d", (long long)dim, kMostHeadDim);
    REQUIRE(eps >= 0.0f && isfinite(eps), "eps=%g", (double)eps);
    if (rope && rope->rot_dim != 0) {
        REQUIRE(rope->rot_dim > 0 && rope->rot_dim <= dim && rope->rot_dim % 2 == 0, "rot_dim=%d: even, 0..head_dim", rope->rot_dim);
        REQUIRE(rope->pairs == GEMM_ROPE_HALVES || rope->pairs == GEMM_ROPE_NEIGHBOURS, "pairs %d", rope->pairs);
        TRY(check_size("rows of the table", rope->rows));
        TRY(check_ld("ld of the table", rope->ld, rope->rot_dim / 2));
        if (tokens > 0 && q_heads + k_heads > 0) {
            REQUIRE(rope->positions, "positions is NULL");
            REQUIRE(rope->rows == 0 || (rope->cos && rope->sin), "cos or sin is NULL");
        }
        p->pos = rope->positions;
        p->cos = rope->cos;
        p->sin = rope->sin;
        p->ldt = rope->ld;
        p->table = rope->rows;
        p->rot = rope->rot_dim;
        p->neighbours = rope->pairs == GEMM_ROPE_NEIGHBOURS;
    }
    p->w[0] = static_cast<const char*>(wq);
    p->w[1] = static_cast<const char*>(wk);
    p->w_type = w_type;
    p->tokens = tokens;
    p->heads[0] = (int)q_heads;
    p->heads[1] = (int)k_heads;
    p->dim = (int)dim;
    p->eps = eps;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_linear(gemm_dtype_t in_type, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* W,
                          int64_t ldw, const void* bias, gemm_dtype_t bias_type, gemm_act_t act, const void* R, int64_t ldr,
                          void* Z, int64_t ldz, void* C, gemm_dtype_t c_type, int64_t ldc, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
    op_clear_error();
    TRY(check_linear(in_type, act, M, N, K));
    REQUIRE(c_type == GEMM_F32 || c_type == in_type, "c_type %d not offered for in_type %d", (int)c_type, (int)in_type);
    REQUIRE(!bias || bias_type == GEMM_F32 || bias_type == in_type, "bias_type %d not offered for in_type %d", (int)bias_type, (int)in_type);
    TRY(check_ld("lda", lda, K));
    TRY(check_ld("ldw", ldw, K));
    TRY(check_ld("ldc", ldc, N));
    if (R) TRY(check_ld("ldr", ldr, N));
    if (Z) TRY(check_ld("ldz", ldz, N));
    TRY(check_ws(workspace));
    if (M == 0 || N == 0) return GEMM_OK;
    REQUIRE(C, "C is NULL");
    REQUIRE(A || K == 0, "A is NULL");
    REQUIRE(W || K == 0, "W is NULL");
    LinearParams p;
    p.A = static_cast<const char*>(A);
    p.W = static_cast<const char*>(W);
    p.bias = static_cast<const char*>(bias);
    p.R = static_cast<const char*>(R);
    p.Z = static_cast<char*>(Z);
    p.C = static_cast<char*>(C);
    p.lda = lda; p.ldw = ldw; p.ldr = R ? ldr : 0; p.ldz = Z ? ldz : 0; p.ldc = ldc;
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.act = act; p.bias_type = bias_type; p.out_type = c_type;
    if (!workspace) workspace_bytes = 0;
    const bool few = linear_few(p, ldw % 64 == 0, workspace_bytes), tiles = !few && linear_tile_fits(p);
    op_note("linear type %d -> %d M=%lld N=%lld K=%lld act=%d: %s", (int)in_type, (int)c_type, (long long)M, (long long)N, (long long)K,
            (int)act, few ? "few rows" : tiles ? "tiles" : "128 x 128 tiles");
    if (few) return launched(launch_linear_skinny(in_type, p, stream));
    return launched(tiles ? launch_linear_tile(in_type, p, workspace, workspace_bytes, stream) : launch_linear_staged(in_type, p, stream));
}

gemm_status_t gemm_linear_workspace_size(gemm_dtype_t in_type, int64_t M, int64_t N, int64_t K, size_t* bytes) {
    op_clear_error();
    REQUIRE(bytes, "bytes is NULL");
    *bytes = 0;
    TRY(check_linear(in_type, GEMM_ACT_NONE, M, N, K));
    if (M > 0 && N > 0 && K > 0) {
        LinearParams p = {};
        p.M = (int)M; p.N = (int)N; p.K = (int)K;
        p.lda = p.ldw = K;   // (of contiguous operands)
        if (!linear_few(p, false, SIZE_MAX) && linear_tile_fits(p)) *bytes = linear_tile_workspace(p);   // (the other kernels use none)
    }
    return GEMM_OK;
}

gemm_status_t gemm_linear_bwd(gemm_dtype_t in_type, int64_t M, int64_t N, int64_t K, gemm_act_t act, const void* dC,
                              gemm_dtype_t dc_type, int64_t lddc, const void* Z, int64_t ldz, const void* A, int64_t lda,
                              const void* W, int64_t ldw, void* dZ, int64_t lddz, void* dA, int64_t ldda, void* dW,
                              gemm_dtype_t dw_type, int64_t lddw, float* dbias, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    op_clear_error();
    TRY(check_linear(in_type, act, M, N, K));
    REQUIRE(dc_type == GEMM_F32 || dc_type == in_type, "dc_type %d not offered for in_type %d", (int)dc_type, (int)in_type);
    REQUIRE(!dW || dw_type == GEMM_F32 || dw_type == in_type, "dw_type %d not offered for in_type %d", (int)dw_type, (int)in_type);
    const bool some = M > 0 && N > 0, same = act == GEMM_ACT_NONE && dc_type == in_type;
    TRY(check_ld("lddc", lddc, N));
    if (act != GEMM_ACT_NONE) TRY(check_ld("ldz", ldz, N));
    if (dZ) TRY(check_ld("lddz", lddz, N));
    if (dA) {
        TRY(check_ld("ldda", ldda, K));
        TRY(check_ld("ldw", ldw, K));
    }
    if (dW) {
        TRY(check_ld("lddw", lddw, K));
        TRY(check_ld("lda", lda, K));
    }
    TRY(check_ws(workspace));
    if (some) {
        REQUIRE(dC, "dC is NULL");
        REQUIRE(Z || act == GEMM_ACT_NONE, "Z is NULL");
        REQUIRE(dZ || same || (!dA && !dW), "dZ is NULL");
        REQUIRE(!dA || W || K == 0, "W is NULL");
        REQUIRE(!dW || A || K == 0, "A is NULL");
    }
    if (!workspace) workspace_bytes = 0;
    if (N == 0 && (!dA || M == 0)) return GEMM_OK;
    const void* dz = dZ ? dZ : dC;
    BackwardPlan b = backward_plan(M, N, K, dz, dZ ? lddz : lddc, A, lda, W, ldw, dA, ldda, in_type, dW, lddw, dw_type, dbias != nullptr, workspace_bytes);
    op_note("linear_bwd type %d M=%lld N=%lld K=%lld act=%d: dZ in %d parts%s%s%s", (int)in_type, (long long)M, (long long)N, (long long)K, (int)act,
            b.parts, b.copies[0].src ? ", dZ copied" : "", b.copies[1].src ? ", A copied" : "", b.copies[2].src ? ", W copied" : "");
    for (const GradParams& f : b.f)
        if (f.C && b.tiles) op_note("  %d x %d x %d: %d x %d tiles, %d splits of the sum", f.M, f.N, f.K, f.bm, f.bn, f.splits);
        else if (f.C) op_note("  %d x %d x %d: as a 16-bit product", f.M, f.N, f.K);
    char* at = static_cast<char*>(workspace) + b.sums;
    for (RowsJob& j : b.copies)
        if (j.src) {
            j.dst = reinterpret_cast<uint8_t*>(at);
            at += round256(j.bytes());
        }
    LinearBwdParams p = {};
    p.dC = static_cast<const char*>(dC);
    p.Z = static_cast<const char*>(Z);
    p.dZ = some ? static_cast<char*>(dZ) : nullptr;
    p.db = dbias;
    p.lddc = lddc; p.ldz = ldz; p.lddz = lddz;
    p.M = M;
    p.N = (int)N;
    p.act = act;
    p.dc_type = dc_type;
    p.part = static_cast<float*>(workspace);
    p.parts = b.parts;
    p.copy = reinterpret_cast<char*>(b.copies[0].dst);
    p.ldcopy = b.copies[0].len_pad / 2;
    p.jobs[0] = b.copies[1];
    p.jobs[1] = b.copies[2];
    if (N > 0 && (dbias || p.dZ || p.copy)) TRY(launched(launch_linear_bwd(in_type, p, stream)));
    else if (p.jobs[0].src || p.jobs[1].src) TRY(launched(launch_rows_pack(p.jobs[0], p.jobs[1], stream)));
    const DbJoin join = {p.part, dbias && b.parts > 1 ? dbias : nullptr, (int)N, b.parts};
    if (b.tiles) {
        auto copied = [](const RowsJob& j, const char* own) { return j.src ? reinterpret_cast<const char*>(j.dst) : own; };
        b.f[0].A = b.f[1].A = copied(b.copies[0], b.f[0].A);
        b.f[1].B = copied(b.copies[1], b.f[1].B);
        b.f[0].B = copied(b.copies[2], b.f[0].B);
        return launched(launch_linear_grad(in_type, b.f, join, at, stream));
    }
    const GradParams none[2] = {};
    TRY(launched(launch_linear_grad(in_type, none, join, nullptr, stream)));
    for (const GradParams& f : b.f)
        if (f.C) TRY(product(in_type, f, static_cast<char*>(workspace) + b.sums, workspace_bytes - b.sums, stream));
    return GEMM_OK;
}

gemm_status_t gemm_linear_bwd_workspace_size(gemm_dtype_t in_type, int64_t M, int64_t N, int64_t K, size_t* bytes) {
    op_clear_error();
    REQUIRE(bytes, "bytes is NULL");
    *bytes = 0;
    TRY(check_linear(in_type, GEMM_ACT_NONE, M, N, K));
    if (M == 0 || N == 0) return GEMM_OK;
    // (contiguous aligned operands, wherever they are, and the larger of dW's types)
    void* at = reinterpret_cast<void*>(uintptr_t(1) << 20);
    const BackwardPlan b = backward_plan(M, N, K, at, N, at, K, at, K, at, K, in_type, at, K, GEMM_F32, true, SIZE_MAX / 2);
    *bytes = b.bytes;
    if (K > 0 && !b.tiles)
        for (const GradParams& f : b.f) {
            size_t more = 0;
            TRY(gemm_workspace_size(in_type, (gemm_dtype_t)f.out_type, f.rows_a ? GEMM_COL_MAJOR : GEMM_ROW_MAJOR, GEMM_ROW_MAJOR, f.M, f.N, f.K,
                                    1.0f, f.A, f.lda, f.B, f.ldb, 0.0f, f.C, f.ldc, nullptr, &more, nullptr));
            *bytes = std::max(*bytes, b.sums + more);
        }
    return GEMM_OK;
}

gemm_status_t gemm_qk_norm_rope(gemm_dtype_t in_type, gemm_dtype_t w_type, int64_t tokens, int64_t q_heads, int64_t k_heads,
                                int64_t head_dim, float eps, const gemm_heads_t* q, const gemm_heads_t* k, const void* wq,
                                const void* wk, const gemm_rope_t* rope, const gemm_heads_t* out_q, const gemm_heads_t* out_k,
                                hipStream_t stream) {
    op_clear_error();
    HeadsParams p;
    TRY(check_qk(in_type, w_type, tokens, q_heads, k_heads, head_dim, eps, wq, wk, rope, &p));
    TRY(check_heads("q", q, tokens, q_heads, head_dim, &p.x[0]));
    TRY(check_heads("k", k, tokens, k_heads, head_dim, &p.x[1]));
    TRY(check_heads("out_q", out_q, tokens, q_heads, head_dim, &p.y[0]));
    TRY(check_heads("out_k", out_k, tokens, k_heads, head_dim, &p.y[1]));
    if (tokens == 0 || q_heads + k_heads == 0) return GEMM_OK;
    op_note("qk_norm_rope type %d tokens=%lld heads=%lld+%lld dim=%lld rot=%d", (int)in_type, (long long)tokens, (long long)q_heads,
            (long long)k_heads, (long long)head_dim, p.rot);
    return launched(launch_heads(in_type, p, stream));
}

gemm_status_t gemm_qk_norm_rope_bwd(gemm_dtype_t in_type, gemm_dtype_t w_type, int64_t tokens, int64_t q_heads, int64_t k_heads,
                                    int64_t head_dim, float eps, const gemm_heads_t* dq, const gemm_heads_t* dk,
                                    const gemm_heads_t* q, const gemm_heads_t* k, const void* wq, const void* wk,
                                    const gemm_rope_t* rope, const gemm_heads_t* dxq, const gemm_heads_t* dxk, float* dwq,
                                    float* dwk, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    op_clear_error();
    HeadsParams p;
    TRY(check_qk(in_type, w_type, tokens, q_heads, k_heads, head_dim, eps, wq, wk, rope, &p));
    TRY(check_heads("dq", dq, tokens, q_heads, head_dim, &p.dy[0]));
    TRY(check_heads("dk", dk, tokens, k_heads, head_dim, &p.dy[1]));
    TRY(check_heads("q", q, tokens, q_heads, head_dim, &p.x[0]));
    TRY(check_heads("k", k, tokens, k_heads, head_dim, &p.x[1]));
    TRY(check_heads("dxq", dxq, tokens, q_heads, head_dim, &p.y[0]));
    TRY(check_heads("dxk", dxk, tokens, k_heads, head_dim, &p.y[1]));
    TRY(check_ws(workspace));
    if ((tokens == 0 || q_heads + k_heads == 0) && !dwq && !dwk) return GEMM_OK;
    p.dw[0] = dwq;
    p.dw[1] = dwk;
    p.part = static_cast<float*>(workspace);
    p.parts = heads_bwd_parts(in_type, p);
    if (dwq || dwk) {   // (partial sums are needed for dw alone)
        const int64_t fit = workspace ? (int64_t)(workspace_bytes / ((size_t)head_dim * sizeof(float))) : 0;
        p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(p.parts, fit));
    }
    op_note("qk_norm_rope_bwd type %d tokens=%lld heads=%lld+%lld dim=%lld rot=%d in %d parts", (int)in_type, (long long)tokens,
            (long long)q_heads, (long long)k_heads, (long long)head_dim, p.rot, p.parts);
    return launched(launch_heads_bwd(in_type, p, stream));
}

gemm_status_t gemm_qk_norm_rope_bwd_workspace_size(gemm_dtype_t in_type, int64_t tokens, int64_t q_heads, int64_t k_heads,
                                                   int64_t head_dim, size_t* bytes) {
    op_clear_error();
    REQUIRE(bytes, "bytes is NULL");
    *bytes = 0;
    HeadsParams p;
    TRY(check_qk(in_type, in_type, tokens, q_heads, k_heads, head_dim, 0.0f, nullptr, nullptr, nullptr, &p));
    const int parts = heads_bwd_most_parts(p);
    if (parts > 1) *bytes = (size_t)parts * (size_t)head_dim * sizeof(float);
    return GEMM_OK;
}

}  // extern "C"
