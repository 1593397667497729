// ops.hpp -- parameters and launchers of the operators around the products: the
// root-mean-square norm, its backward pass, the product of 8-bit operands with scales and
// the product with 4-bit weights (internal to the library; the entry points are in ops.cpp).
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "libgemm.h"

namespace gemm {

enum : int { DT_F8E4M3 = 3 };   // continues common.hpp's DT_*: OCP 8-bit floats, 4 exponent bits

// Records a status and its text for gemm_last_error() and returns it (libgemm.cpp).
gemm_status_t op_fail(gemm_status_t s, const char* fmt, ...);
void op_clear_error();
void op_note(const char* fmt, ...);   // a line on stderr with GEMM_DEBUG set

// ---------------------------------------------------------------- norm
struct NormParams {
    const char* x;
    const char* r;       // residual added to x, or NULL
    const char* w;       // NULL: ones
    char* h;             // x + r as it is kept, or NULL
    char* y;
    float* scale;        // per row, y_type DT_F8E4M3 only
    float* rstd;         // per row, or NULL
    int64_t ldx, ldr, ldh, ldy;   // elements
    int64_t rows;
    int cols;
    int w_type, y_type;
    float eps;
};
hipError_t launch_norm(int in_type, const NormParams& p, hipStream_t st);

struct NormBwdParams {
    const char* dy;
    const char* h;
    const char* w;       // NULL: ones
    const float* rstd;
    const char* dh;      // gradient added to dx, or NULL
    char* dx;
    float* dw;           // NULL: not computed
    float* part;         // parts x cols partial sums of dw (parts > 1)
    int64_t lddy, ldh, lddh, lddx;
    int64_t rows;
    int cols;
    int w_type;
    int parts;           // workgroups, each a fixed set of rows and one partial row of dw
    int strip_blocks;    // (the launch's: workgroups that sum dw by columns, before the others)
};
// Rows that one workgroup of the backward kernel works on at a time, and the number of
// workgroups it would like for this problem (its partial sums need parts * cols floats).
int norm_bwd_parts(int in_type, int64_t rows, int cols);
hipError_t launch_norm_bwd(int in_type, const NormBwdParams& p, hipStream_t st);

// ---------------------------------------------------------------- rows into a workspace
// dst: rows_pad rows of len_pad bytes (a multiple of 16), the source's rows of len bytes (ld apart) with zeros behind
// and below; fewer than 2^32 chunks of 16 bytes.  src == NULL: no job.
struct RowsJob {
    const uint8_t* src;
    uint8_t* dst;
    int64_t ld, rows, len, rows_pad, len_pad;
    int64_t bytes() const { return rows_pad * len_pad; }
};
hipError_t launch_rows_pack(const RowsJob& a, const RowsJob& b, hipStream_t st);

// ---------------------------------------------------------------- 8-bit product
struct F8Params {
    const uint8_t* A;    // M x K, K contiguous
    const uint8_t* B;    // N x K, K contiguous
    char* C;
    const float* sa;     // per row of A, or NULL (ones)
    const float* sb;     // per row of B, or NULL (ones)
    int64_t lda, ldb, ldc;
    int M, N, K;
    float alpha, beta;
    int out_type;
};
constexpr int kF8SkinnyRows = 32;   // rows of A that launch_f8_skinny takes
double f8_skinny_us(const F8Params& p);              // what either is expected to take with so few rows
double f8_tile_us(const F8Params& p, size_t ws_bytes);
hipError_t launch_f8_skinny(const F8Params& p, hipStream_t st);
bool f8_tile_fits(const F8Params& p);
size_t f8_tile_workspace(const F8Params& p);   // of a product that fits
hipError_t launch_f8_tile(const F8Params& p, void* ws, size_t ws_bytes, hipStream_t st);
hipError_t launch_f8_staged(const F8Params& p, hipStream_t st);

// ---------------------------------------------------------------- 4-bit weights
struct W4Params {
    const char* A;       // M x K, bf16 or f16
    const uint8_t* W;    // N rows of ceil(K/2) bytes
    const char* scales;  // N x groups, A's type
    const char* zeros;   // the same, or NULL (8)
    char* C;
    int64_t lda, ldw, lds, ldc;   // elements; ldw in bytes
    int M, N, K, group;
    float alpha, beta;
    int out_type;
};
constexpr int kW4VectorRows = 4;    // rows of A that launch_w4_vector takes
hipError_t launch_w4_vector(int in_type, const W4Params& p, hipStream_t st);
double w4_skinny_us(const W4Params& p);                // what either is expected to take
double w4_tile_us(const W4Params& p, size_t ws_bytes);
bool w4_tile_fits(const W4Params& p, size_t ws_bytes);
size_t w4_tile_workspace(int64_t M, int64_t N, int64_t K, int64_t group);
hipError_t launch_w4_tile(int in_type, const W4Params& p, void* ws, size_t ws_bytes, hipStream_t st);
hipError_t launch_w4_skinny(int in_type, const W4Params& p, hipStream_t st);

// ---------------------------------------------------------------- product with bias, activation and residual
struct LinearParams {
    const char* A;       // M x K, K contiguous, 16 bits
    const char* W;       // N x K, the same
    const char* bias;    // N, or NULL
    const char* R;       // M x N of C's type, added behind the activation, or NULL
    char* Z;             // M x N of A's type: the sums with their bias, or NULL
    char* C;
    int64_t lda, ldw, ldr, ldz, ldc;   // elements
    int M, N, K;
    int act, bias_type, out_type;
};
constexpr int kLinearSkinnyRows = 32;   // rows of A that launch_linear_skinny takes
hipError_t launch_linear_skinny(int in_type, const LinearParams& p, hipStream_t st);
bool linear_tile_fits(const LinearParams& p);
size_t linear_tile_workspace(const LinearParams& p);   // of a product that fits
hipError_t launch_linear_tile(int in_type, const LinearParams& p, void* ws, size_t ws_bytes, hipStream_t st);
hipError_t launch_linear_staged(int in_type, const LinearParams& p, hipStream_t st);

// The backward pass's first launch: dZ = dC * act'(Z), its sums over the rows, and copies of rows.
struct LinearBwdParams {
    const char* dC;      // M x N
    const char* Z;       // M x N, or NULL (act 0)
    char* dZ;            // M x N, or NULL (dC is it)
    char* copy;          // dZ in aligned rows of whole 16 bytes, zeros behind N, or NULL
    float* db;           // N, or NULL
    float* part;         // parts x N partial sums of db (parts > 1)
    int64_t lddc, ldz, lddz, ldcopy;
    int64_t M;
    int N;
    int act, dc_type;
    int parts;           // what the rows are cut into
    RowsJob jobs[2];
};
int linear_bwd_parts(int64_t M, int64_t N);   // parts that the pass would like
hipError_t launch_linear_bwd(int in_type, const LinearBwdParams& p, hipStream_t st);

// C = A B, the products of the backward pass: B is K x N row by row; A is M x K row by row, or (rows_a) K x M row by row.
struct GradParams {
    const char* A;
    const char* B;
    char* C;             // NULL: not wanted
    int64_t lda, ldb, ldc;   // elements
    int M, N, K;
    bool rows_a;
    int out_type;
    size_t ws;           // what it uses of a workspace, as planned
    int bm, bn, splits;
};
bool linear_grad_fits(const GradParams& p);
// Tiles and splits of both products ([0] with A along the sum, [1] with rows_a) and what their splits' sums need.
void linear_grad_plan(GradParams (&p)[2], size_t ws_bytes);
// The sums of db's parts, which ride in the last launch.
struct DbJoin {
    const float* part;
    float* db;           // NULL: nothing to join
    int N, parts;
};
hipError_t launch_linear_grad(int in_type, const GradParams (&p)[2], const DbJoin& db, void* ws, hipStream_t st);

// ---------------------------------------------------------------- norm and rotation of heads
struct HeadsTensor {
    const char* p;
    int64_t ld, hs;      // elements between tokens, between heads
};
struct HeadsParams {     // [0]: queries, [1]: keys
    HeadsTensor x[2];
    HeadsTensor dy[2];   // backward only
    HeadsTensor y[2];    // what is written: y, or dx
    const char* w[2];    // NULL: ones
    float* dw[2];        // backward: NULL where not wanted
    float* part;         // backward: parts x dim partial sums of dw (parts > 1)
    const int64_t* pos;
    const float* cos;
    const float* sin;
    int64_t ldt, table;  // the table's rows: floats apart, how many
    int64_t tokens;
    int heads[2];
    int dim, rot, neighbours;
    int w_type;
    float eps;
    int parts;
};
constexpr int kMostHeadDim = 1024;
hipError_t launch_heads(int in_type, const HeadsParams& p, hipStream_t st);
int heads_bwd_most_parts(const HeadsParams& p);
int heads_bwd_parts(int in_type, const HeadsParams& p);   // in_type: DT_*
hipError_t launch_heads_bwd(int in_type, const HeadsParams& p, hipStream_t st);

}  // namespace gemm
