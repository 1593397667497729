"""Torch-tensor form of the operators around the products: the root-mean-square norm and its
backward pass (also through autograd), the product of 8-bit operands and the product with 4-bit
weights (which have none); and of a transformer block's dense parts, with their backward passes: the
product with bias, activation and residual, and the norm of queries and keys with the rotation by position.

As ``libgemm.matmul``, these only read shapes, strides and pointers; every step on the
GPU runs in the library's kernels, and there is no fallback.  Calls may be captured into graphs; a
backward pass through autograd with its forward pass, from leaves that no graph made before still
holds (torch ties a leaf's gradient to that one's stream, which a capture must not meet).  Inputs with forward-mode
tangents are refused.  ``quantize_f8`` and ``quantize_w4`` prepare weights once, in plain torch, on any device.
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


class _Running(lg.Running):
    """No operator has a forward-mode derivative, and kernels that read a dual tensor's memory would lose its tangent."""
    tangents = False


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

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, residual, act, out_dtype, workspace):
            keep = act != "none" and any(ctx.needs_input_grad[:3])
            y, z = _linear(x, weight, bias, act, residual, out_dtype, keep, workspace)
            ctx.save_for_backward(x, weight, z)
            ctx.act, ctx.bias = act, bias.dtype if bias is not None else None
            return y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            x, weight, z = ctx.saved_tensors
            of_x, of_weight, of_bias, of_residual = ctx.needs_input_grad[:4]
            dx = dw = db = None
            if of_x or of_weight or of_bias:
                dx, dw, db = linear_backward(dy.contiguous(), x, weight, z, ctx.act, (of_x, of_weight, of_bias))
            return dx, dw, db.to(ctx.bias) if of_bias else None, dy if of_residual else None, None, None, None

    class Heads(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk, positions, cos, sin, pairs, eps):
            ctx.save_for_backward(q, k, wq, wk, positions, cos, sin)
            ctx.pairs, ctx.eps = pairs, eps
            return _qk_norm_rope(q, k, wq, wk, positions, cos, sin, pairs, eps)

        @staticmethod
        @once_differentiable
        def backward(ctx, dq, dk):
            q, k, wq, wk, positions, cos, sin = ctx.saved_tensors
            of_q, of_k, of_wq, of_wk = ctx.needs_input_grad[:4]
            gq, gk, gwq, gwk = qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), q, k, wq, wk, positions, cos, sin, ctx.pairs,
                                                     ctx.eps, of_wq or of_wk)
            return (gq if of_q else None, gk if of_k else None, gwq.to(wq.dtype) if of_wq else None,
                    gwk.to(wk.dtype) if of_wk else None, None, None, None, None, None)

    class NoBackward(torch.autograd.Function):
        @staticmethod
        def forward(ctx, name, result, *inputs):
            ctx.name = name
            ctx.mark_dirty(result)
            return result

        @staticmethod
        def backward(ctx, _):
            raise RuntimeError(f"{ctx.name} has no backward pass: detach its inputs")

    return Norm, NoBackward, Linear, Heads


def rmsnorm(x, weight=None, residual=None, eps: float = 1e-6, out_dtype=None, stream=None) -> RmsNorm:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, row by row, in `out_dtype`
    (x's by default; torch.float8_e4m3fn gives codes and a scale per row).  Gradients of y (not of
    8-bit codes) and h reach x, weight and residual through ``rmsnorm_backward``."""
    if not _wants_gradient(x, weight, residual):
        return _rmsnorm(x, weight, residual, eps, out_dtype, stream)
    with _Running(stream, x.device, x, weight, residual) as on:   # (its backward pass runs on the same stream)
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
    with _Running(stream, x.device, x, weight, residual) as on:
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
    with _Running(stream, h.device, dy, h, weight, rstd, dh, workspace) as on:
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
    with _Running(stream, a.device, a, b, scale_a, scale_b, C, workspace) as on:
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
    with _Running(stream, a.device, a, codes, scales, zeros, C, workspace) as on:
        C, ldc = _result(on, C, M, N, beta, out_dtype or a.dtype, a.device)
        held, ws, nbytes = _workspace(workspace, lambda: lg.gemm_w4_workspace_size(code, M, N, K, group), a.device)
        lg.check(lg.gemm_w4(code, M, N, K, group, alpha, a.data_ptr(), lda, codes.data_ptr(), ldw, scales.data_ptr(),
                            zeros.data_ptr() if zeros is not None else 0, lds, beta, C.data_ptr(), _code(C.dtype), ldc, ws,
                            nbytes, on.handle))
        return _no_gradient("matmul_w4", C, a, codes, scales, zeros)


ACTS = {"none": lg.GEMM_ACT_NONE, "relu": lg.GEMM_ACT_RELU, "gelu": lg.GEMM_ACT_GELU, "gelu_tanh": lg.GEMM_ACT_GELU_TANH,
        "silu": lg.GEMM_ACT_SILU}
PAIRS = {"halves": lg.GEMM_ROPE_HALVES, "neighbours": lg.GEMM_ROPE_NEIGHBOURS}


def _one_of(table, name: str, value) -> int:
    if value not in table:
        raise ValueError(f"{name} {value!r}: one of {', '.join(table)}")
    return table[value]


def linear(x, weight, bias=None, act: str = "none", residual=None, out_dtype=None, workspace="auto", stream=None):
    """act(x weight^T + bias) + residual; x: M x K and weight: N x K in bf16 or f16; the result, and residual with it, in
    their type (the default) or fp32; act: "none", "relu", "gelu", "gelu_tanh" or "silu".  Gradients reach
    x, weight, bias and residual through ``linear_backward``."""
    if not _wants_gradient(x, weight, bias, residual):
        return _linear(x, weight, bias, act, residual, out_dtype, False, workspace, stream)[0]
    with _Running(stream, x.device, x, weight, bias, residual, workspace) as on:   # (its backward pass runs on the same stream)
        y = _functions()[2].apply(x, weight, bias, residual, act, out_dtype, workspace)
        on.keep(y)
    return y


def linear_keeping(x, weight, bias=None, act: str = "none", residual=None, out_dtype=None, workspace="auto", stream=None):
    """(``linear``'s result, z = x weight^T + bias in x's type, which ``linear_backward`` reads); without autograd."""
    return _linear(x, weight, bias, act, residual, out_dtype, True, workspace, stream)


def _linear(x, weight, bias, act, residual, out_dtype, keep, workspace, stream=None):
    import torch
    lda, ldw = _rows(x, "x"), _rows(weight, "weight", None, x.dtype, x.device)
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"shapes {tuple(x.shape)} and {tuple(weight.shape)}: rows of different lengths")
    code, out_dtype, a = _code(x.dtype), out_dtype or x.dtype, _one_of(ACTS, "act", act)
    c_code = _code(out_dtype)
    b = _vector(bias, "bias", N, (x.dtype, torch.float32), x.device)
    ldr = _rows(residual, "residual", (M, N), out_dtype, x.device) if residual is not None else 0
    with _Running(stream, x.device, x, weight, bias, residual, workspace) as on:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
        z = torch.empty((M, N), dtype=x.dtype, device=x.device) if keep else None
        on.keep(y, z)
        held, ws, nbytes = _workspace(workspace, lambda: lg.gemm_linear_workspace_size(code, M, N, K), x.device)
        lg.check(lg.gemm_linear(code, M, N, K, x.data_ptr(), lda, weight.data_ptr(), ldw, b, _code(bias.dtype) if b else 0, a,
                                residual.data_ptr() if ldr else 0, ldr, z.data_ptr() if keep else 0, max(N, 1), y.data_ptr(), c_code,
                                max(N, 1), ws, nbytes, on.handle))
    return y, z


def linear_backward(dy, x, weight, z=None, act: str = "none", need=(True, True, True), dw_dtype=None, workspace="auto", stream=None):
    """(dx, dw, db) of ``linear`` from its z (None for act "none"); dx in x's type, dw in weight's or `dw_dtype`
    (fp32), db in fp32; `need`: which of them are wanted (None for the others).  residual's gradient is dy."""
    import torch
    lda, ldw = _rows(x, "x"), _rows(weight, "weight", None, x.dtype, x.device)
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"shapes {tuple(x.shape)} and {tuple(weight.shape)}: rows of different lengths")
    code, a = _code(x.dtype), _one_of(ACTS, "act", act)
    lddy = _rows(dy, "dy", (M, N), None, x.device)
    if z is None and act != "none":
        raise ValueError(f"act {act!r} needs z")
    ldz = _rows(z, "z", (M, N), x.dtype, x.device) if act != "none" else 0
    with _Running(stream, x.device, dy, x, weight, z, workspace) as on:
        new = lambda wanted, *shape, dtype: torch.empty(shape, dtype=dtype, device=x.device) if wanted else None  # noqa: E731
        dx, dw = new(need[0], M, K, dtype=x.dtype), new(need[1], N, K, dtype=dw_dtype or weight.dtype)
        db = new(need[2], N, dtype=torch.float32)
        dz = new((need[0] or need[1]) and (act != "none" or dy.dtype != x.dtype), M, N, dtype=x.dtype)
        on.keep(dx, dw, db)
        held, ws, nbytes = _workspace(workspace, lambda: lg.gemm_linear_bwd_workspace_size(code, M, N, K), x.device)
        at = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
        lg.check(lg.gemm_linear_bwd(code, M, N, K, a, dy.data_ptr(), _code(dy.dtype), lddy, at(z) if ldz else 0, ldz, x.data_ptr(), lda,
                                    weight.data_ptr(), ldw, at(dz), max(N, 1), at(dx), max(K, 1), at(dw),
                                    _code(dw.dtype) if need[1] else 0, max(K, 1), at(db), ws, nbytes, on.handle))
    return dx, dw, db


def _heads(t, name: str, shape=None, dtype=None, device=None):
    """Checks tokens x heads x dim with contiguous heads and gives what the library reads of it."""
    if t.dim() != 3 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}" + (f", not {tuple(shape)}" if shape is not None else ", not tokens x heads x dim"))
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, not {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return lg.GemmHeads(t.data_ptr(), t.stride(0), t.stride(1))


def _rope(positions, cos, sin, pairs, tokens, device):
    import torch
    code = _one_of(PAIRS, "pairs", pairs)
    if positions is None and cos is None and sin is None:
        return None
    if positions is None or cos is None or sin is None:
        raise ValueError("positions, cos and sin come together")
    at = _vector(positions, "positions", tokens, torch.int64, device)
    ld = _rows(cos, "cos", None, torch.float32, device)
    if _rows(sin, "sin", cos.shape, torch.float32, device) != ld:
        raise ValueError("sin: the row stride of cos")
    return lg.GemmRope(at, cos.data_ptr(), sin.data_ptr(), ld, cos.shape[0], 2 * cos.shape[1], code)


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, device=None):
    """(cos, sin), rows x rot_dim / 2 each in fp32, of the angles position * base^(-2 i / rot_dim), taken in 64 bits."""
    import torch
    if rows < 0 or rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rows {rows}, rot_dim {rot_dim}: not negative, rot_dim even")
    rate = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * rate
    return angle.cos().float(), angle.sin().float()


def qk_norm_rope(q, k, wq=None, wk=None, positions=None, cos=None, sin=None, pairs: str = "halves", eps: float = 1e-6, stream=None):
    """(q, k), each head divided by the root of its mean square, times wq or wk, and its first 2 * cos.shape[1] elements turned by
    the token's position.  q, k: tokens x heads x dim, any strides with contiguous heads; positions: int64, a row of
    cos and sin (``rope_table``) each; pairs: element i with i + half of those that turn ("halves") or 2 i with 2 i + 1 ("neighbours").
    Without positions, cos and sin: the norm alone.  Gradients reach q, k, wq and wk through ``qk_norm_rope_backward``."""
    if _wants_gradient(cos, sin):
        raise ValueError("no gradient reaches cos and sin: detach them")
    if not _wants_gradient(q, k, wq, wk):
        return _qk_norm_rope(q, k, wq, wk, positions, cos, sin, pairs, eps, stream)
    with _Running(stream, q.device, q, k, wq, wk, positions, cos, sin) as on:   # (its backward pass runs on the same stream)
        out = _functions()[3].apply(q, k, wq, wk, positions, cos, sin, pairs, eps)
        on.keep(*out)
    return out


def _qk(q, k, wq, wk):
    """What both passes check of their inputs: (types' codes, weights' addresses)"""
    import torch
    if k.dim() != 3 or q.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
        raise ValueError(f"q and k: shapes {tuple(q.shape)} and {tuple(k.shape)}, not tokens x heads x dim with tokens and dim alike")
    if wq is not None and wk is not None and wq.dtype != wk.dtype:
        raise ValueError(f"wq and wk: {wq.dtype} and {wk.dtype}")
    w = wq if wq is not None else wk
    at = [_vector(t, name, q.shape[2], (q.dtype, torch.float32), q.device) for t, name in ((wq, "wq"), (wk, "wk"))]
    return _code(q.dtype), _code(w.dtype) if w is not None else 0, at


def _qk_norm_rope(q, k, wq, wk, positions, cos, sin, pairs, eps, stream=None):
    import torch
    code, w_code, w = _qk(q, k, wq, wk)
    tokens, heads, dim = q.shape
    qh, kh = _heads(q, "q"), _heads(k, "k", None, q.dtype, q.device)
    rope = _rope(positions, cos, sin, pairs, tokens, q.device)
    with _Running(stream, q.device, q, k, wq, wk, positions, cos, sin) as on:
        out = [torch.empty(t.shape, dtype=q.dtype, device=q.device) for t in (q, k)]
        on.keep(*out)
        lg.check(lg.gemm_qk_norm_rope(code, w_code, tokens, heads, k.shape[1], dim, eps, qh, kh, *w, rope, *(_heads(t, "") for t in out),
                                      on.handle))
    return tuple(out)


def qk_norm_rope_backward(dq, dk, q, k, wq=None, wk=None, positions=None, cos=None, sin=None, pairs: str = "halves", eps: float = 1e-6,
                          need_dw: bool = True, workspace="auto", stream=None):
    """(gradients of q, of k, of wq, of wk) of ``qk_norm_rope`` from those of its results and its inputs; the weights' in
    fp32 (None unless `need_dw`, which without a workspace leaves one workgroup for all)."""
    import torch
    code, w_code, w = _qk(q, k, wq, wk)
    tokens, heads, dim = q.shape
    given = [_heads(dq, "dq", q.shape, q.dtype, q.device), _heads(dk, "dk", k.shape, q.dtype, q.device), _heads(q, "q"),
             _heads(k, "k", None, q.dtype, q.device)]
    rope = _rope(positions, cos, sin, pairs, tokens, q.device)
    with _Running(stream, q.device, dq, dk, q, k, wq, wk, positions, cos, sin, workspace) as on:
        dx = [torch.empty(t.shape, dtype=q.dtype, device=q.device) for t in (q, k)]
        dw = [torch.empty(dim, dtype=torch.float32, device=q.device) if need_dw else None for _ in range(2)]
        on.keep(*dx, *dw)
        held, ws, nbytes = _workspace(workspace if need_dw else None,
                                      lambda: lg.gemm_qk_norm_rope_bwd_workspace_size(code, tokens, heads, k.shape[1], dim), q.device)
        lg.check(lg.gemm_qk_norm_rope_bwd(code, w_code, tokens, heads, k.shape[1], dim, eps, *given, *w, rope,
                                          *(_heads(t, "") for t in dx), *(t.data_ptr() if need_dw else 0 for t in dw), ws, nbytes, on.handle))
    return (*dx, *dw)


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
