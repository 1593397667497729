"""ctypes binding of libgemm.so -- argument marshalling only.

The functions named like the C ABI (``gemm_f32``, ``gemm_bf16``, ``gemm_f16``, their
``_ex`` forms, ``gemm_plan``, ``gemm_schedule``, ``gemm_status_string``,
``gemm_last_error``) take plain integers for device pointers and return the status
code.  ``matmul`` is a convenience wrapper over torch tensors: it reads the layout and
leading dimension of each operand from its strides and passes ``data_ptr()`` and the
current HIP stream; every step of the computation runs in the library's kernels.

There is no fallback: if libgemm.so cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libgemm.so")

GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_HIP = 0, 1, 2, 3
GEMM_ROW_MAJOR, GEMM_COL_MAJOR = 0, 1
GEMM_F32, GEMM_BF16, GEMM_F16, GEMM_F8E4M3 = 0, 1, 2, 3
(GEMM_KERNEL_AUTO, GEMM_KERNEL_VALU_RING, GEMM_KERNEL_VALU_STAGED, GEMM_KERNEL_MFMA_RING,
 GEMM_KERNEL_MFMA_STAGED, GEMM_KERNEL_SCALE) = range(6)
(GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_GELU_TANH, GEMM_ACT_SILU) = range(5)
GEMM_ROPE_HALVES, GEMM_ROPE_NEIGHBOURS = 0, 1
GEMM_FLAG_NO_XCD_REMAP = 1
GEMM_FLAG_EQUAL_LDS = 2
GEMM_FLAG_POISON_LDS = 4
GEMM_MAX_NSTAGE = 4
GEMM_STATIC_WS_BYTES = 33554432
GEMM_CEIL_THREADS = 512
GEMM_CEIL_FRAG_ELEMS = 16384
GEMM_CEIL_MAX_GRID = 65536

KERNEL_NAMES = {0: "none", 1: "valu_ring", 2: "valu_staged", 3: "mfma_ring", 4: "mfma_staged", 5: "scale"}

# Symbols declared in include/libgemm.h.
EXPORTS = ("gemm_f32", "gemm_bf16", "gemm_f16", "gemm_f32_ex", "gemm_bf16_ex", "gemm_f16_ex",
           "gemm_bf16_ws", "gemm_f16_ws", "gemm_ws_static", "gemm_workspace_size", "gemm_plan", "gemm_tune", "gemm_tune_ws",
           "gemm_schedule", "gemm_pipe_copy", "gemm_mfma_ceiling", "gemm_h2d_staged", "gemm_h2d_staged_async", "gemm_status_string",
           "gemm_last_error", "gemm_rmsnorm", "gemm_rmsnorm_bwd", "gemm_rmsnorm_bwd_workspace_size", "gemm_f8",
           "gemm_f8_workspace_size", "gemm_w4", "gemm_w4_workspace_size", "gemm_linear", "gemm_linear_workspace_size",
           "gemm_linear_bwd", "gemm_linear_bwd_workspace_size", "gemm_qk_norm_rope", "gemm_qk_norm_rope_bwd",
           "gemm_qk_norm_rope_bwd_workspace_size")


class GemmOpts(ctypes.Structure):
    _fields_ = [("nstage", ctypes.c_int), ("kernel", ctypes.c_int), ("tile", ctypes.c_int),
                ("flags", ctypes.c_int)]


class GemmPlan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("nstage", ctypes.c_int), ("tile", ctypes.c_int),
                ("bm", ctypes.c_int), ("bn", ctypes.c_int), ("bk", ctypes.c_int),
                ("threads", ctypes.c_int), ("lds_bytes", ctypes.c_int), ("grid", ctypes.c_int64),
                ("packed", ctypes.c_int)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel_name"] = KERNEL_NAMES.get(self.kernel, str(self.kernel))
        return d


class GemmHeads(ctypes.Structure):
    """tokens x heads x head_dim elements by their address and strides (elements)."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class GemmRope(ctypes.Structure):
    """The rotation by position: addresses of positions, cos and sin, the table's pitch and rows, rot_dim, pairs."""
    _fields_ = [("positions", ctypes.c_void_p), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("rot_dim", ctypes.c_int), ("pairs", ctypes.c_int)]


class GemmError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_name(status)}: {msg}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load():
    """Load libgemm.so (built in-tree by ``tiled_stage_software_amd.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        i64, vp, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        base = [i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp]
        lib.gemm_f32.argtypes = base + [i64, vp]
        lib.gemm_f32_ex.argtypes = base + [i64, vp, ctypes.POINTER(GemmOpts)]
        for name in ("gemm_bf16", "gemm_f16"):
            getattr(lib, name).argtypes = base + [i32, i64, vp]
            getattr(lib, name + "_ex").argtypes = base + [i32, i64, vp, ctypes.POINTER(GemmOpts)]
            getattr(lib, name + "_ws").argtypes = base + [i32, i64, vp, ctypes.POINTER(GemmOpts), vp,
                                                          ctypes.c_size_t]
        for name in ("gemm_f32", "gemm_bf16", "gemm_f16", "gemm_f32_ex", "gemm_bf16_ex", "gemm_f16_ex",
                     "gemm_bf16_ws", "gemm_f16_ws"):
            getattr(lib, name).restype = i32
        lib.gemm_ws_static.argtypes = [i32] + base + [i32, i64, vp, ctypes.POINTER(GemmOpts)]
        lib.gemm_ws_static.restype = i32
        lib.gemm_workspace_size.argtypes = [i32, i32, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp,
                                            i64, ctypes.POINTER(GemmOpts), ctypes.POINTER(ctypes.c_size_t),
                                            ctypes.POINTER(GemmPlan)]
        lib.gemm_workspace_size.restype = i32
        lib.gemm_plan.argtypes = [i32, i32, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                  ctypes.POINTER(GemmOpts), ctypes.POINTER(GemmPlan)]
        lib.gemm_plan.restype = i32
        lib.gemm_schedule.argtypes = [i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int), i32]
        lib.gemm_schedule.restype = i32
        lib.gemm_tune.argtypes = [i32, i32, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                  vp, i32, ctypes.POINTER(GemmOpts), ctypes.POINTER(ctypes.c_float)]
        lib.gemm_tune.restype = i32
        lib.gemm_tune_ws.argtypes = [i32, i32, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                     vp, vp, ctypes.c_size_t, i32, ctypes.POINTER(GemmOpts),
                                     ctypes.POINTER(ctypes.c_float)]
        lib.gemm_tune_ws.restype = i32
        lib.gemm_pipe_copy.argtypes = [vp, vp, i64, i32, vp]
        lib.gemm_pipe_copy.restype = i32
        lib.gemm_mfma_ceiling.argtypes = [i32, i32, vp, vp, i64, i64, vp]
        lib.gemm_mfma_ceiling.restype = i32
        for name in ("gemm_h2d_staged", "gemm_h2d_staged_async"):
            getattr(lib, name).argtypes = [vp, vp, i64, vp, i64, i32, vp]
            getattr(lib, name).restype = i32
        sz, szp = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        lib.gemm_rmsnorm.argtypes = [i32, i32, i32, i64, i64, f32, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp]
        lib.gemm_rmsnorm_bwd.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, sz, vp]
        lib.gemm_rmsnorm_bwd_workspace_size.argtypes = [i32, i64, i64, szp]
        lib.gemm_f8.argtypes = [i64, i64, i64, f32, vp, i64, vp, vp, i64, vp, f32, vp, i32, i64, vp, sz, vp]
        lib.gemm_f8_workspace_size.argtypes = [i64, i64, i64, szp]
        lib.gemm_w4.argtypes = [i32, i64, i64, i64, i64, f32, vp, i64, vp, i64, vp, vp, i64, f32, vp, i32, i64, vp, sz, vp]
        lib.gemm_w4_workspace_size.argtypes = [i32, i64, i64, i64, i64, szp]
        lib.gemm_linear.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, vp, i32, i32, vp, i64, vp, i64, vp, i32, i64, vp, sz, vp]
        lib.gemm_linear_workspace_size.argtypes = [i32, i64, i64, i64, szp]
        lib.gemm_linear_bwd.argtypes = [i32, i64, i64, i64, i32, vp, i32, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i32,
                                        i64, vp, vp, sz, vp]
        lib.gemm_linear_bwd_workspace_size.argtypes = [i32, i64, i64, i64, szp]
        hp, rp = ctypes.POINTER(GemmHeads), ctypes.POINTER(GemmRope)
        lib.gemm_qk_norm_rope.argtypes = [i32, i32, i64, i64, i64, i64, f32, hp, hp, vp, vp, rp, hp, hp, vp]
        lib.gemm_qk_norm_rope_bwd.argtypes = [i32, i32, i64, i64, i64, i64, f32, hp, hp, hp, hp, vp, vp, rp, hp, hp, vp, vp, vp, sz, vp]
        lib.gemm_qk_norm_rope_bwd_workspace_size.argtypes = [i32, i64, i64, i64, i64, szp]
        for name in ("gemm_rmsnorm", "gemm_rmsnorm_bwd", "gemm_rmsnorm_bwd_workspace_size", "gemm_f8",
                     "gemm_f8_workspace_size", "gemm_w4", "gemm_w4_workspace_size", "gemm_linear", "gemm_linear_workspace_size",
                     "gemm_linear_bwd", "gemm_linear_bwd_workspace_size", "gemm_qk_norm_rope", "gemm_qk_norm_rope_bwd",
                     "gemm_qk_norm_rope_bwd_workspace_size"):
            getattr(lib, name).restype = i32
        lib.gemm_status_string.argtypes = [i32]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_last_error.argtypes = []
        lib.gemm_last_error.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _opts(nstage=0, kernel=0, tile=0, flags=0) -> Optional[GemmOpts]:
    if not (nstage or kernel or tile or flags):
        return None
    return GemmOpts(int(nstage), int(kernel), int(tile), int(flags))


def _ref(o):
    return ctypes.byref(o) if o is not None else None


# ------------------------------------------------------------------ C ABI names

def gemm_f32(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f32(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0) -> int:
    return load().gemm_bf16(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream)


def gemm_f16(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0) -> int:
    return load().gemm_f16(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream)


def gemm_f32_ex(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0, opts=None) -> int:
    return load().gemm_f32_ex(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, _ref(opts))


def gemm_bf16_ex(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0, opts=None) -> int:
    return load().gemm_bf16_ex(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream, _ref(opts))


def gemm_f16_ex(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0, opts=None) -> int:
    return load().gemm_f16_ex(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream, _ref(opts))


def gemm_bf16_ws(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0, opts=None,
                 workspace=0, workspace_bytes=0) -> int:
    return load().gemm_bf16_ws(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream, _ref(opts),
                               workspace, workspace_bytes)


def gemm_f16_ws(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0, opts=None,
                workspace=0, workspace_bytes=0) -> int:
    return load().gemm_f16_ws(la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream, _ref(opts),
                              workspace, workspace_bytes)


def gemm_ws_static(in_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream=0, opts=None) -> int:
    """gemm_bf16_ws / gemm_f16_ws with the library's static workspace (allocates nothing)."""
    return load().gemm_ws_static(in_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, c_type, ldc, stream,
                                 _ref(opts))


def gemm_workspace_size(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, opts=None):
    """Returns (status, bytes, GemmPlan of the call given that many bytes)."""
    n = ctypes.c_size_t(0)
    plan = GemmPlan()
    s = load().gemm_workspace_size(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                   _ref(opts), ctypes.byref(n), ctypes.byref(plan))
    return s, n.value, plan


def gemm_plan(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, opts=None):
    """Returns (status, GemmPlan)."""
    plan = GemmPlan()
    s = load().gemm_plan(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                         _ref(opts), ctypes.byref(plan))
    return s, plan


def gemm_schedule(kernel, nstage, num_k, ksteps):
    """Event list [(type, slab, slot, arg), ...] of the kernel family's K loop, or None."""
    lib = load()
    n = lib.gemm_schedule(kernel, nstage, num_k, ksteps, None, 0)
    if n < 0:
        return None
    buf = (ctypes.c_int * (4 * max(n, 1)))()
    lib.gemm_schedule(kernel, nstage, num_k, ksteps, buf, n)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


def gemm_tune(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0, reps=10):
    """(status, GemmOpts of the fastest variant, its ms per call) -- see include/libgemm.h."""
    best = GemmOpts()
    ms = ctypes.c_float(0.0)
    s = load().gemm_tune(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, reps,
                         ctypes.byref(best), ctypes.byref(ms))
    return s, best, ms.value


def gemm_tune_ws(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0,
                 workspace=0, workspace_bytes=0, reps=10):
    """gemm_tune for the workspace entry points: (status, GemmOpts, ms per call)."""
    best = GemmOpts()
    ms = ctypes.c_float(0.0)
    s = load().gemm_tune_ws(in_type, c_type, la, lb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream,
                            workspace, workspace_bytes, reps, ctypes.byref(best), ctypes.byref(ms))
    return s, best, ms.value


def gemm_pipe_copy(dst: int, src: int, nbytes: int, nstage: int = 0, stream: int = 0) -> int:
    """dst[0, nbytes) = src[0, nbytes) through the nStage LDS ring (device pointers)."""
    return load().gemm_pipe_copy(dst, src, nbytes, nstage, stream)


def gemm_mfma_ceiling(in_type: int, shape: int, frags: int, sums: int, grid: int, iters: int,
                      stream: int = 0) -> int:
    """Matrix instructions on register operands (device pointers): grid * 8 * iters * 2^20
    FLOPs; one fp32 accumulator sum per thread into sums."""
    return load().gemm_mfma_ceiling(in_type, shape, frags, sums, grid, iters, stream)


def gemm_h2d_staged(dst: int, src: int, nbytes: int, staging: int, chunk_bytes: int, nstage: int = 2,
                    stream: int = 0) -> int:
    """dst (device) = src (pageable host) through nstage page-locked staging slots."""
    return load().gemm_h2d_staged(dst, src, nbytes, staging, chunk_bytes, nstage, stream)


def gemm_h2d_staged_async(dst: int, src: int, nbytes: int, staging: int, chunk_bytes: int, nstage: int = 2,
                          stream: int = 0) -> int:
    """gemm_h2d_staged returning before the last DMAs finish (sync `stream` before reusing staging)."""
    return load().gemm_h2d_staged_async(dst, src, nbytes, staging, chunk_bytes, nstage, stream)


def gemm_rmsnorm(in_type, w_type, y_type, rows, cols, eps, x, ldx, r, ldr, w, h, ldh, y, ldy, scale, rstd, stream=0) -> int:
    """h = x + r; y = h * rstd * w, for GEMM_F8E4M3 with a scale per row (see include/libgemm.h)."""
    return load().gemm_rmsnorm(in_type, w_type, y_type, rows, cols, eps, x, ldx, r, ldr, w, h, ldh, y, ldy, scale, rstd,
                               stream)


def gemm_rmsnorm_bwd(in_type, w_type, rows, cols, dy, lddy, h, ldh, w, rstd, dh, lddh, dx, lddx, dw, workspace=0,
                     workspace_bytes=0, stream=0) -> int:
    return load().gemm_rmsnorm_bwd(in_type, w_type, rows, cols, dy, lddy, h, ldh, w, rstd, dh, lddh, dx, lddx, dw,
                                   workspace, workspace_bytes, stream)


def gemm_f8(M, N, K, alpha, A, lda, scale_a, B, ldb, scale_b, beta, C, c_type, ldc, workspace=0, workspace_bytes=0,
            stream=0) -> int:
    """C = alpha * diag(scale_a) A B^T diag(scale_b) + beta * C, A and B e4m3."""
    return load().gemm_f8(M, N, K, alpha, A, lda, scale_a, B, ldb, scale_b, beta, C, c_type, ldc, workspace,
                          workspace_bytes, stream)


def gemm_w4(in_type, M, N, K, group, alpha, A, lda, codes, ldw, scales, zeros, lds, beta, C, c_type, ldc, workspace=0,
            workspace_bytes=0, stream=0) -> int:
    """C = alpha * A W^T + beta * C, W in 4-bit codes with group scales."""
    return load().gemm_w4(in_type, M, N, K, group, alpha, A, lda, codes, ldw, scales, zeros, lds, beta, C, c_type, ldc,
                          workspace, workspace_bytes, stream)


def _size_of(fn, *args):
    n = ctypes.c_size_t(0)
    s = fn(*args, ctypes.byref(n))
    return s, n.value


def gemm_rmsnorm_bwd_workspace_size(in_type, rows, cols):
    """(status, bytes)"""
    return _size_of(load().gemm_rmsnorm_bwd_workspace_size, in_type, rows, cols)


def gemm_f8_workspace_size(M, N, K):
    """(status, bytes)"""
    return _size_of(load().gemm_f8_workspace_size, M, N, K)


def gemm_w4_workspace_size(in_type, M, N, K, group):
    """(status, bytes)"""
    return _size_of(load().gemm_w4_workspace_size, in_type, M, N, K, group)


def gemm_linear(in_type, M, N, K, A, lda, W, ldw, bias, bias_type, act, R, ldr, Z, ldz, C, c_type, ldc, workspace=0,
                workspace_bytes=0, stream=0) -> int:
    """C = act(A W^T + bias) + R; Z = A W^T + bias where it is wanted (see include/libgemm.h)."""
    return load().gemm_linear(in_type, M, N, K, A, lda, W, ldw, bias, bias_type, act, R, ldr, Z, ldz, C, c_type, ldc, workspace,
                              workspace_bytes, stream)


def gemm_linear_bwd(in_type, M, N, K, act, dC, dc_type, lddc, Z, ldz, A, lda, W, ldw, dZ, lddz, dA, ldda, dW, dw_type, lddw, dbias,
                    workspace=0, workspace_bytes=0, stream=0) -> int:
    return load().gemm_linear_bwd(in_type, M, N, K, act, dC, dc_type, lddc, Z, ldz, A, lda, W, ldw, dZ, lddz, dA, ldda, dW, dw_type,
                                  lddw, dbias, workspace, workspace_bytes, stream)


def gemm_qk_norm_rope(in_type, w_type, tokens, q_heads, k_heads, head_dim, eps, q, k, wq, wk, rope, out_q, out_k, stream=0) -> int:
    """Norm of each head of q and k with the rotation by position; q, k, out_q, out_k: GemmHeads, rope: GemmRope or None."""
    return load().gemm_qk_norm_rope(in_type, w_type, tokens, q_heads, k_heads, head_dim, eps, q, k, wq, wk, rope, out_q, out_k, stream)


def gemm_qk_norm_rope_bwd(in_type, w_type, tokens, q_heads, k_heads, head_dim, eps, dq, dk, q, k, wq, wk, rope, dxq, dxk, dwq, dwk,
                          workspace=0, workspace_bytes=0, stream=0) -> int:
    return load().gemm_qk_norm_rope_bwd(in_type, w_type, tokens, q_heads, k_heads, head_dim, eps, dq, dk, q, k, wq, wk, rope, dxq, dxk,
                                        dwq, dwk, workspace, workspace_bytes, stream)


def gemm_linear_workspace_size(in_type, M, N, K):
    """(status, bytes)"""
    return _size_of(load().gemm_linear_workspace_size, in_type, M, N, K)


def gemm_linear_bwd_workspace_size(in_type, M, N, K):
    """(status, bytes)"""
    return _size_of(load().gemm_linear_bwd_workspace_size, in_type, M, N, K)


def gemm_qk_norm_rope_bwd_workspace_size(in_type, tokens, q_heads, k_heads, head_dim):
    """(status, bytes)"""
    return _size_of(load().gemm_qk_norm_rope_bwd_workspace_size, in_type, tokens, q_heads, k_heads, head_dim)


def gemm_status_string(s: int) -> str:
    return load().gemm_status_string(int(s)).decode()


def gemm_last_error() -> str:
    return load().gemm_last_error().decode()


def status_name(s: int) -> str:
    try:
        return gemm_status_string(s)
    except Exception:  # library not loadable: still give the number
        return f"status {s}"


def check(status: int):
    if status != GEMM_OK:
        raise GemmError(status, gemm_last_error())


# ------------------------------------------------------------------ torch convenience

class Running:
    """The device and the stream that a call's kernels run on (a handle; None: the current one),
    as torch's current ones while the call lasts.  Handle 0 is every device's default stream, so a
    launch would else run on whichever device is current.  What the call allocates comes from that
    stream's memory, not from blocks that earlier work of the caller's stream may still use.  The
    tensors that the call is given are marked for that stream, and by ``keep`` its results for the
    caller's: either may be dropped at once."""
    tangents = True   # False: inputs with forward-mode tangents are refused (``requires_grad`` says nothing of those)

    def __init__(self, stream, device, *given):
        import torch
        if not self.tangents and getattr(torch.autograd.forward_ad, "_current_level", 0) >= 0:   # (hardly ever: a question takes 0.3 us)
            for t in given:
                if isinstance(t, torch.Tensor) and torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
                    raise NotImplementedError("the operators have no forward-mode derivatives: detach their inputs")
        if device.type != "cuda":
            raise ValueError(f"tensors on {device}: the kernels run on the GPU")
        self.caller = torch.cuda.current_stream(device)
        self.handle = self.caller.cuda_stream if stream is None else stream
        self.device = torch.cuda.device(device) if device.index != torch.cuda.current_device() else None
        self.other = None
        if self.handle != self.caller.cuda_stream:
            runs = torch.cuda.ExternalStream(self.handle, device=device)
            self.other = torch.cuda.stream(runs)
            for t in given:
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(runs)

    def __enter__(self):
        if self.device is not None:
            self.device.__enter__()
        if self.other is not None:
            self.other.__enter__()
        return self

    def __exit__(self, *error):
        if self.other is not None:
            self.other.__exit__(*error)
        if self.device is not None:
            self.device.__exit__(*error)

    def keep(self, *tensors):
        if self.other is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.caller)


def workspace_of(t, device):
    """(pointer, bytes) of a tensor that serves as workspace: whole memory, as the call uses every
    byte from its first on."""
    if t.device != device:
        raise ValueError(f"workspace is on {t.device}, not {device}")
    if not t.is_contiguous():
        raise ValueError("workspace: a contiguous tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def _layout_of(t, rows, cols):
    """(layout, ld) of a 2-D tensor view, or None if it is neither row- nor column-major."""
    s0, s1 = t.stride()
    if cols == 1 and rows == 1:
        return GEMM_ROW_MAJOR, 1
    if s1 == 1 and (rows == 1 or s0 >= cols):
        return GEMM_ROW_MAJOR, max(s0, cols) if rows > 1 else cols
    if s0 == 1 and (cols == 1 or s1 >= rows):
        return GEMM_COL_MAJOR, max(s1, rows) if cols > 1 else rows
    return None


def matmul(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, out_dtype=None, stream=None,
           nstage: int = 0, kernel: int = 0, tile: int = 0, flags: int = 0, workspace=None):
    """C = alpha*A@B + beta*C on device tensors (A: M x K, B: K x N, any of the two
    layouts per operand, C row-major).  Returns C.  16-bit inputs: `workspace` (a device
    tensor, 256-byte aligned, at least gemm_workspace_size bytes; "auto" = allocate one
    with torch) lets the direct ring take operands it cannot read in place."""
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shapes {tuple(A.shape)} @ {tuple(B.shape)}")
    if A.dtype != B.dtype:
        raise ValueError("A and B must have the same dtype")
    M, K = A.shape
    N = B.shape[1]
    la = _layout_of(A, M, K)
    lb = _layout_of(B, K, N)
    if la is None or lb is None:
        raise ValueError("operands must be row- or column-major views")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
    elif C.dim() != 2 or tuple(C.shape) != (M, N) or (N > 1 and C.stride(1) != 1):
        raise ValueError("C must be an M x N row-major view")
    elif M > 1 and C.stride(0) < N:
        # an expanded or row-overlapping view: the kernels would write past its storage
        raise ValueError(f"C rows overlap (stride {C.stride(0)} < N = {N})")
    with Running(stream, A.device, A, B, C, workspace) as on:
        if C is None:
            C = torch.empty((M, N), dtype=A.dtype if out_dtype is None else out_dtype, device=A.device)
            on.keep(C)
        ldc = C.stride(0) if M > 1 else max(N, 1)
        st = on.handle
        o = _opts(nstage, kernel, tile, flags)
        if A.dtype == torch.float32:
            if C.dtype != torch.float32:
                raise ValueError("fp32 inputs give fp32 C")
            s = gemm_f32_ex(la[0], lb[0], M, N, K, alpha, A.data_ptr(), la[1], B.data_ptr(), lb[1],
                            beta, C.data_ptr(), ldc, st, o)
        elif A.dtype in (torch.bfloat16, torch.float16):
            ct = {torch.float32: GEMM_F32, torch.bfloat16: GEMM_BF16, torch.float16: GEMM_F16}[C.dtype]
            if workspace is None:
                fn = gemm_bf16_ex if A.dtype == torch.bfloat16 else gemm_f16_ex
                s = fn(la[0], lb[0], M, N, K, alpha, A.data_ptr(), la[1], B.data_ptr(), lb[1],
                       beta, C.data_ptr(), ct, ldc, st, o)
            else:
                if isinstance(workspace, str):
                    if workspace != "auto":
                        raise ValueError("workspace: a device tensor or 'auto'")
                    it = GEMM_BF16 if A.dtype == torch.bfloat16 else GEMM_F16
                    s, nbytes, _ = gemm_workspace_size(it, ct, la[0], lb[0], M, N, K, alpha, A.data_ptr(), la[1],
                                                       B.data_ptr(), lb[1], beta, C.data_ptr(), ldc, o)
                    check(s)
                    workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=A.device)
                fn = gemm_bf16_ws if A.dtype == torch.bfloat16 else gemm_f16_ws
                s = fn(la[0], lb[0], M, N, K, alpha, A.data_ptr(), la[1], B.data_ptr(), lb[1],
                       beta, C.data_ptr(), ct, ldc, st, o, *workspace_of(workspace, A.device))
        else:
            raise ValueError(f"unsupported dtype {A.dtype}")
        check(s)
    return C


def gemm_operands(in_dtype: str, out_dtype: str, la, lb, M, N, K, alpha, A_ptr, lda, B_ptr, ldb,
                  beta, C_ptr, ldc, stream=0, nstage=0, kernel=0, tile=0, flags=0, ws_ptr=0, ws_bytes=0) -> int:
    """Dispatch on dtype names ('f32' / 'bf16' / 'f16') with raw pointers (16-bit inputs
    with ws_ptr != 0: the workspace entry points)."""
    o = _opts(nstage, kernel, tile, flags)
    if in_dtype == "f32":
        return gemm_f32_ex(la, lb, M, N, K, alpha, A_ptr, lda, B_ptr, ldb, beta, C_ptr, ldc, stream, o)
    ct = {"f32": GEMM_F32, "bf16": GEMM_BF16, "f16": GEMM_F16}[out_dtype]
    if ws_ptr:
        fn = gemm_bf16_ws if in_dtype == "bf16" else gemm_f16_ws
        return fn(la, lb, M, N, K, alpha, A_ptr, lda, B_ptr, ldb, beta, C_ptr, ct, ldc, stream, o, ws_ptr, ws_bytes)
    fn = gemm_bf16_ex if in_dtype == "bf16" else gemm_f16_ex
    return fn(la, lb, M, N, K, alpha, A_ptr, lda, B_ptr, ldb, beta, C_ptr, ct, ldc, stream, o)
