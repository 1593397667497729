"""Torch-tensor form of the operators around the products: the root-mean-square norm and its
backward pass (also through autograd), the product of 8-bit operands and the product with 4-bit
weights (which have none).

As ``libgemm.matmul``, these only read shapes, strides and pointers; every step on the
GPU runs in the library's kernels, and there is no fallback.  ``quantize_f8`` and
``quantize_w4`` prepare weights once, in plain torch, on any device.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

from . import libgemm as lg

F8_MAX = 448.0          # the largest finite e4m3 value
TINY = 2.0 ** -126      # the least scale: a row of zeros has it


class RmsNorm(NamedTuple):
    """What ``rmsnorm`` returns: y; its scale per row (8-bit y, else None); h = x + residual
    (x itself where there is no residual); rstd, which the backward pass reads."""
    y: "torch.Tensor"
    scale: Optional["torch.Tensor"]
    h: "torch.Tensor"
    rstd: "torch.Tensor"


def _code(dtype) -> int:
    import torch
    codes = {torch.float32: lg.GEMM_F32, torch.bfloat16: lg.GEMM_BF16, torch.float16: lg.GEMM_F16,
             torch.float8_e4m3fn: lg.GEMM_F8E4M3}
    if dtype not in codes:
        raise ValueError(f"unsupported dtype {dtype}")
    return codes[dtype]


def _rows(t, name: str, shape=None, dtype=None, device=None) -> int:
    """Checks a 2-D tensor with contiguous rows and gives its leading dimension."""
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}" + (f", not {tuple(shape)}" if shape is not None else ""))
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, not {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: rows overlap (stride {t.stride(0)} < {cols})")
    return max(t.stride(0), cols, 1) if rows > 1 else max(cols, 1)


def _vector(t, name: str, n: int, dtype, device) -> int:
    if t is None:
        return 0
    if t.dim() != 1 or t.numel() != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: a contiguous vector of {n}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name}: {t.dtype}")
    return t.data_ptr()


def _workspace(workspace, size, device):
    """(tensor, pointer, bytes) of a workspace: None, a device tensor, or "auto" (allocated here)."""
    import torch
    if workspace is None:
        return None, 0, 0
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace: None, a device tensor or 'auto'")
        s, nbytes = size()
        lg.check(s)
        if not nbytes:
            return None, 0, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace, *lg.workspace_of(workspace, device)


def _wants_gradient(*tensors) -> bool:
    import torch
    return torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in tensors)


@functools.lru_cache(maxsize=None)
def _functions():
    """(the norm as autograd has it, the mark of a result that no gradient passes)."""
    import torch
    from torch.autograd.function import once_differentiable

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, residual, eps, out_dtype):
            n = _rmsnorm(x, weight, residual, eps, out_dtype)
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(n.h, weight, n.rstd)
            ctx.mark_non_differentiable(*(t for t in (n.rstd, n.scale) if t is not None), *([n.y] if n.scale is not None else []))
            return n.y, n.scale, n.h if residual is not None else None, n.rstd

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, _scale, dh, _rstd):
            h, weight, rstd = ctx.saved_tensors
            of_x, of_weight, of_residual = ctx.needs_input_grad[:3]
            if dy is None:
                return dh if of_x else None, None, dh if of_residual else None, None, None
            rows = lambda t, dtype: t.to(dtype).contiguous() if t is not None else None  # noqa: E731
            wide = h.dtype if dy.dtype == h.dtype else torch.float32   # (a y of another type: nothing is rounded on the way in)
            w = weight if weight is None or weight.dtype == wide else weight.float()
            dx, dw = rmsnorm_backward(rows(dy, wide), h if wide == h.dtype else h.float(), w, rstd, rows(dh, wide), of_weight)
            dx = dx.to(h.dtype)
            return (dx if of_x else None, dw.to(weight.dtype) if of_weight else None, dx if of_residual else None, None, None)

    class NoBackward(torch.autograd.Function):
        @staticmethod
        def forward(ctx, name, result, *inputs):
            ctx.name = name
            ctx.mark_dirty(result)
            return result

        @staticmethod
        def backward(ctx, _):
            raise RuntimeError(f"{ctx.name} has no backward pass: detach its inputs")

    return Norm, NoBackward


def rmsnorm(x, weight=None, residual=None, eps: float = 1e-6, out_dtype=None, stream=None) -> RmsNorm:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, row by row, in `out_dtype`
    (x's by default; torch.float8_e4m3fn gives codes and a scale per row).  Gradients of y (not of
    8-bit codes) and h reach x, weight and residual through ``rmsnorm_backward``."""
    if not _wants_gradient(x, weight, residual):
        return _rmsnorm(x, weight, residual, eps, out_dtype, stream)
    with lg.Running(stream, x.device, x, weight, residual) as on:   # (its backward pass runs on the same stream)
        y, scale, h, rstd = _functions()[0].apply(x, weight, residual, eps, out_dtype)
        on.keep(y, scale, h, rstd)
    return RmsNorm(y, scale, x if h is None else h, rstd)


def _rmsnorm(x, weight=None, residual=None, eps: float = 1e-6, out_dtype=None, stream=None) -> RmsNorm:
    import torch
    ldx = _rows(x, "x")
    rows, cols = x.shape
    out_dtype = out_dtype or x.dtype
    w = _vector(weight, "weight", cols, (x.dtype, torch.float32), x.device)
    y_code = _code(out_dtype)
    ldr = _rows(residual, "residual", x.shape, x.dtype, x.device) if residual is not None else 0
    with lg.Running(stream, x.device, x, weight, residual) as on:
        h, ldh = x, 0
        if ldr:
            h, ldh = torch.empty((rows, cols), dtype=x.dtype, device=x.device), max(cols, 1)
        y = torch.empty((rows, cols), dtype=out_dtype, device=x.device)
        scale = torch.empty(rows, device=x.device) if y_code == lg.GEMM_F8E4M3 else None
        rstd = torch.empty(rows, device=x.device)
        on.keep(h if ldr else None, y, scale, rstd)
        lg.check(lg.gemm_rmsnorm(_code(x.dtype), _code(weight.dtype) if w else 0, y_code, rows, cols, eps, x.data_ptr(), ldx,
                                 residual.data_ptr() if ldr else 0, ldr, w, h.data_ptr() if ldh else 0, ldh, y.data_ptr(),
                                 max(cols, 1), scale.data_ptr() if scale is not None else 0, rstd.data_ptr(), on.handle))
    return RmsNorm(y, scale, h, rstd)


def rmsnorm_backward(dy, h, weight, rstd, dh=None, need_dw: bool = True, workspace="auto", stream=None):
    """(dx, dw) of ``rmsnorm`` from its h and rstd; dh (or None) is the gradient that reaches
    h by other paths and is added to dx; dw is fp32 (None unless `need_dw`)."""
    import torch
    ldh = _rows(h, "h")
    rows, cols = h.shape
    lddy = _rows(dy, "dy", h.shape, h.dtype, h.device)
    lddh = _rows(dh, "dh", h.shape, h.dtype, h.device) if dh is not None else 0
    w = _vector(weight, "weight", cols, (h.dtype, torch.float32), h.device)
    r = _vector(rstd, "rstd", rows, torch.float32, h.device)
    with lg.Running(stream, h.device, dy, h, weight, rstd, dh, workspace) as on:
        dx = torch.empty((rows, cols), dtype=h.dtype, device=h.device)
        dw = torch.empty(cols, device=h.device) if need_dw else None
        on.keep(dx, dw)
        held, ws, nbytes = _workspace(workspace if need_dw else None,
                                      lambda: lg.gemm_rmsnorm_bwd_workspace_size(_code(h.dtype), rows, cols), h.device)
        lg.check(lg.gemm_rmsnorm_bwd(_code(h.dtype), _code(weight.dtype) if w else 0, rows, cols, dy.data_ptr(), lddy,
                                     h.data_ptr(), ldh, w, r, dh.data_ptr() if lddh else 0, lddh, dx.data_ptr(),
                                     max(cols, 1), dw.data_ptr() if need_dw else 0, ws, nbytes, on.handle))
    return dx, dw


def _no_gradient(name, C, *inputs):
    """C; where an input (or the C that was added to) wants a gradient, one whose backward pass says that there is none."""
    return _functions()[1].apply(name, C, *inputs) if _wants_gradient(C, *inputs) else C


def _result(on, C, M, N, beta, out_dtype, device):
    """(C, its leading dimension) of a product."""
    import torch
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((M, N), dtype=out_dtype, device=device)
        on.keep(C)
    return C, _rows(C, "C", (M, N), None, device)


def matmul_f8(a, b, scale_a=None, scale_b=None, C=None, alpha: float = 1.0, beta: float = 0.0, out_dtype=None,
              workspace="auto", stream=None):
    """C = alpha * diag(scale_a) a b^T diag(scale_b) + beta * C; a: M x K and b: N x K in
    float8_e4m3fn; C in fp32, bf16 (the default) or f16."""
    import torch
    lda, ldb = _rows(a, "a", None, torch.float8_e4m3fn), _rows(b, "b", None, torch.float8_e4m3fn, a.device)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)}: rows of different lengths")
    sa = _vector(scale_a, "scale_a", M, torch.float32, a.device)
    sb = _vector(scale_b, "scale_b", N, torch.float32, a.device)
    with lg.Running(stream, a.device, a, b, scale_a, scale_b, C, workspace) as on:
        C, ldc = _result(on, C, M, N, beta, out_dtype or torch.bfloat16, a.device)
        held, ws, nbytes = _workspace(workspace, lambda: lg.gemm_f8_workspace_size(M, N, K), a.device)
        lg.check(lg.gemm_f8(M, N, K, alpha, a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb, beta, C.data_ptr(), _code(C.dtype),
                            ldc, ws, nbytes, on.handle))
        return _no_gradient("matmul_f8", C, a, b, scale_a, scale_b)


def matmul_w4(a, codes, scales, zeros=None, group: int = 128, C=None, alpha: float = 1.0, beta: float = 0.0,
              out_dtype=None, workspace="auto", stream=None):
    """C = alpha * a W^T + beta * C, W[n][k] = scales[n][k // group] * (code[n][k] - zeros[n][k // group])
    (8 without zeros); codes: N x ceil(K/2) bytes, an even k in the low half; a: bf16 or
    f16; C in a's type (the default) or fp32."""
    import torch
    lda = _rows(a, "a")
    M, K = a.shape
    N = codes.shape[0]
    groups = -(-K // group) if group > 0 else 0
    ldw = _rows(codes, "codes", (N, (K + 1) // 2), torch.uint8, a.device)
    lds = _rows(scales, "scales", (N, groups), a.dtype, a.device)
    if zeros is not None and _rows(zeros, "zeros", (N, groups), a.dtype, a.device) != lds:
        raise ValueError("zeros: the row stride of scales")
    code = _code(a.dtype)
    with lg.Running(stream, a.device, a, codes, scales, zeros, C, workspace) as on:
        C, ldc = _result(on, C, M, N, beta, out_dtype or a.dtype, a.device)
        held, ws, nbytes = _workspace(workspace, lambda: lg.gemm_w4_workspace_size(code, M, N, K, group), a.device)
        lg.check(lg.gemm_w4(code, M, N, K, group, alpha, a.data_ptr(), lda, codes.data_ptr(), ldw, scales.data_ptr(),
                            zeros.data_ptr() if zeros is not None else 0, lds, beta, C.data_ptr(), _code(C.dtype), ldc, ws,
                            nbytes, on.handle))
        return _no_gradient("matmul_w4", C, a, codes, scales, zeros)


def quantize_f8(t):
    """(codes, scale per row) of a 2-D tensor in float8_e4m3fn."""
    import torch
    v = t.float()
    scale = (v.abs().amax(1) / F8_MAX).clamp_min(TINY)
    return (v / scale[:, None]).to(torch.float8_e4m3fn), scale


def quantize_w4(w, group: int = 128, dtype=None, zeros: bool = False):
    """(codes, scales, zeros or None) of an N x K weight for ``matmul_w4``; scales in `dtype`
    (w's by default).  Without zeros the codes are centred on 8, with them they run from a group's
    least value, or zero, to its largest, or zero: a zero point is then a whole number from 0 to
    15, which any type holds."""
    import torch
    if group < 32 or group % 32:
        raise ValueError(f"group {group}: a multiple of 32")
    N, K = w.shape
    dtype = dtype or w.dtype
    groups = -(-K // group)
    v = torch.zeros(N, groups * group, device=w.device)
    v[:, :K] = w.float()
    v = v.view(N, groups, group)
    least = torch.finfo(dtype).tiny
    if zeros:
        low, high = v.amin(2).clamp_max(0), v.amax(2).clamp_min(0)
        scales = ((high - low) / 15).clamp_min(least).to(dtype)
        zero = (-low / scales.float()).round().clamp(0, 15).to(dtype)
    else:
        scales = (v.abs().amax(2) / 7.5).clamp_min(least).to(dtype)
        zero = torch.full_like(scales, 8.0)
    q = (v / scales.float()[:, :, None] + zero.float()[:, :, None]).round().clamp(0, 15).to(torch.uint8)
    q = q.view(N, groups * group)[:, :K]
    if K % 2:
        q = torch.cat([q, torch.zeros_like(q[:, :1])], 1)
    return (q[:, 0::2] | q[:, 1::2] << 4).contiguous(), scales, zero if zeros else None
