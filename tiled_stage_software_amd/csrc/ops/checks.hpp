// checks.hpp -- argument checks of the operators' entry points.
#pragma once

#include "ops.hpp"

namespace gemm {

constexpr int64_t kMaxSize = int64_t(1) << 30;
constexpr int64_t kWsAlign = 256;

#define REQUIRE(cond, ...)                                                   \
    do {                                                                     \
        if (!(cond)) return op_fail(GEMM_ERR_INVALID_ARG, __VA_ARGS__);      \
    } while (0)

inline bool float_type(int t) { return t == GEMM_F32 || t == GEMM_BF16 || t == GEMM_F16; }

inline gemm_status_t check_size(const char* what, int64_t v) {
    REQUIRE(v >= 0 && v <= kMaxSize, "%s=%lld: sizes are 0..2^30", what, (long long)v);
    return GEMM_OK;
}
inline gemm_status_t check_ld(const char* what, int64_t ld, int64_t least) {
    REQUIRE(ld >= 1 && ld >= least, "%s=%lld < %lld", what, (long long)ld, (long long)least);
    return GEMM_OK;
}
inline gemm_status_t check_ws(const void* ws) {
    REQUIRE(reinterpret_cast<uintptr_t>(ws) % kWsAlign == 0, "workspace must be %lld-byte aligned", (long long)kWsAlign);
    return GEMM_OK;
}
#define TRY(expr)                              \
    do {                                       \
        const gemm_status_t s_ = (expr);       \
        if (s_ != GEMM_OK) return s_;          \
    } while (0)

inline gemm_status_t launched(hipError_t e) {
    if (e != hipSuccess) return op_fail(GEMM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return GEMM_OK;
}

}  // namespace gemm
