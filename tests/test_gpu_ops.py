"""The operators around the products on the GPU against plain 64-bit forms.

Tolerances count roundings: half a step of the output's type, and for fp32 sums the
worst case of one rounding (2^-24 of the terms' magnitudes) per term on the longest way."""
import pytest
import torch

from gpu_util import DEV, say
from ops_util import (DT, U32, f8_64, f8_cut, norm64, norm_bwd64, norm_steps, off, padded, rounding, untouched, w4_64)
from tiled_stage_software_amd import libgemm as lg, ops

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lg.load()  # fails loudly if the library is missing
    torch.zeros(1, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def code(t):
    return {torch.float32: lg.GEMM_F32, torch.bfloat16: lg.GEMM_BF16, torch.float16: lg.GEMM_F16,
            torch.float8_e4m3fn: lg.GEMM_F8E4M3}[t.dtype]


# ------------------------------------------------------------------ norm

def run_norm(x, r, w, out, pad=0, lead=0, eps=EPS, want_h=True):
    """gemm_rmsnorm on rows `pad` elements apart; checks that nothing else is written."""
    rows, cols = x.shape
    X, _ = padded(x, pad, DEV, lead=lead)
    R = padded(r, pad, DEV, lead=lead)[0] if r is not None else None
    W = w.to(DEV) if w is not None else None
    y, yw = padded(torch.zeros(rows, cols, dtype=out), pad, DEV, lead=lead)
    h, hw = padded(torch.zeros(rows, cols, dtype=x.dtype), pad, DEV, lead=lead)
    scale = torch.full((rows,), -7.0, device=DEV)
    rstd = torch.full((rows,), -7.0, device=DEV)
    lg.check(lg.gemm_rmsnorm(code(X), code(W) if W is not None else 0, code(y), rows, cols, eps, X.data_ptr(), X.stride(0),
                             R.data_ptr() if R is not None else 0, X.stride(0), W.data_ptr() if W is not None else 0,
                             h.data_ptr() if want_h else 0, h.stride(0), y.data_ptr(), y.stride(0), scale.data_ptr(),
                             rstd.data_ptr(), torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert untouched(y, yw) and untouched(h, hw)
    if out != torch.float8_e4m3fn:
        assert bool((scale == -7.0).all())
    if not want_h:
        assert bool((h.float() == 0).all())
    return y.cpu(), scale.cpu(), h.cpu(), rstd.cpu()


def check_norm(x, r, w, out, **kw):
    y, scale, h, rstd = run_norm(x, r, w, out, **kw)
    h64, rstd64, y64 = norm64(x, r, w, kw.get("eps", EPS))
    if kw.get("want_h", True):
        assert torch.equal(h.view(torch.uint8), h64.view(torch.uint8))
    # the sum is off by at most `steps` roundings, the root halves that; a few more for the
    # division, the root, the products by rstd and by w
    rel = (norm_steps(x.shape[1]) / 2 + 8) * U32
    assert off(rstd, rstd64, rel * rstd64) <= 1
    if out == torch.float8_e4m3fn:
        s64 = (y64.abs().amax(1) / ops.F8_MAX).clamp_min(ops.TINY)
        assert off(scale, s64, (rel + 4 * U32) * s64) <= 1
        q64 = y64 / s64[:, None]
        back, allowed = y.double(), rounding(q64, out) + (2 * rel + 8 * U32) * q64.abs()
        e = off(back, q64, allowed)
    else:
        e = off(y, y64, rounding(y64, out) + rel * y64.abs())
    assert e <= 1, e
    return e


NORM_SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (4, 512), (7, 513), (9, 1000), (3, 1025), (2, 2048), (6, 2049),
               (3, 4001), (2, 8192), (1, 8200), (2, 16385), (2, 33000)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_norm(rows, cols, t):
    g = gen(rows * 100003 + cols)
    x = torch.randn(rows, cols, generator=g).to(DT[t])
    r = (2 * torch.randn(rows, cols, generator=g)).to(DT[t])
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(DT[t])
    worst = [check_norm(x, r, w, DT[t]), check_norm(x, r, w, DT["f8"], pad=3, lead=1),
             check_norm(x, None, w.float(), DT["f8"]), check_norm(x, None, None, DT["f32"], pad=8, want_h=False),
             check_norm(x, r, w.float(), DT["bf16"], pad=1, lead=3)]
    say(f"[norm] {t} {rows}x{cols}: {max(worst):.3f} of the tolerance")


@pytest.mark.parametrize("cols", [40, 1000, 4096, 40000])
def test_norm_special_rows(cols):
    """Zeros, one value, values near the type's ends, infinities and NaN stay in their rows."""
    t = torch.bfloat16
    g = gen(cols)
    x = torch.randn(9, cols, generator=g).to(t)
    x[1] = 0
    x[2] = 0
    x[2, cols // 2] = -3.0
    x[3] = 2.0 ** -100                 # its square underflows: rstd is 1 / sqrt(eps)
    x[4, cols - 1] = float("nan")
    x[5, 0] = float("inf")
    x[6] = 2.0 ** 60
    x[7, cols // 3] = -float("inf")
    w = torch.ones(cols, dtype=t)
    y, scale, h, rstd = run_norm(x, None, w, torch.float8_e4m3fn)
    assert torch.equal(h.view(torch.int16), x.view(torch.int16))
    assert bool((y[1].float() == 0).all()) and float(scale[1]) == ops.TINY
    assert float(y[2].float().min()) == -448.0 and int((y[2].float() != 0).sum()) == 1
    for bad in (4, 5, 7):
        assert not bool(torch.isfinite(y[bad].float() * scale[bad]).any())
    for fine in (0, 1, 2, 3, 6, 8):
        assert bool(torch.isfinite(y[fine].float()).all()) and bool(torch.isfinite(scale[fine]))
    keep = [0, 1, 2, 6, 8]
    check_norm(x[keep], None, w, torch.float8_e4m3fn)
    check_norm(x[keep], None, w, torch.float32)
    y32, _, _, r32 = run_norm(x, None, w, torch.float32)
    assert bool(torch.isnan(y32[4]).all()) and bool(torch.isnan(y32[5, 0])) and bool((y32[5, 1:] == 0).all())
    assert off(r32[3:4], torch.tensor([1e3]), torch.tensor([1.0])) <= 1


def test_norm_of_a_kept_sum_is_the_same():
    """Adding the residual first and norming the kept h later gives the same bits."""
    g = gen(5)
    x = torch.randn(33, 4096, generator=g).bfloat16().to(DEV)
    r = torch.randn(33, 4096, generator=g).bfloat16().to(DEV)
    w = torch.randn(4096, generator=g).bfloat16().to(DEV)
    one = ops.rmsnorm(x, w, r, out_dtype=torch.float8_e4m3fn)
    two = ops.rmsnorm(one.h, w, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(one.y.view(torch.uint8), two.y.view(torch.uint8))
    assert torch.equal(one.scale, two.scale) and torch.equal(one.rstd, two.rstd)
    assert two.h.data_ptr() == one.h.data_ptr()


@pytest.mark.parametrize("cols", [300, 5000, 40000])
def test_norm_in_place(cols):
    g = gen(cols)
    x0 = torch.randn(17, cols, generator=g).bfloat16()
    r0 = torch.randn(17, cols, generator=g).bfloat16()
    w = torch.randn(cols, generator=g).bfloat16().to(DEV)
    want = ops.rmsnorm(x0.to(DEV), w, r0.to(DEV))
    x, r = x0.to(DEV), r0.to(DEV)
    rstd = torch.empty(17, device=DEV)
    lg.check(lg.gemm_rmsnorm(lg.GEMM_BF16, lg.GEMM_BF16, lg.GEMM_BF16, 17, cols, EPS, x.data_ptr(), cols, r.data_ptr(), cols,
                             w.data_ptr(), r.data_ptr(), cols, x.data_ptr(), cols, 0, rstd.data_ptr(),
                             torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(r, want.h) and torch.equal(x, want.y) and torch.equal(rstd, want.rstd)


# ------------------------------------------------------------------ norm, backward

def check_bwd(dy, h, w, rstd, dh, pad=0, lead=0, workspace="auto", need_dw=True):
    rows, cols = h.shape
    view = lambda t: padded(t, pad, DEV, lead=lead)[0] if t is not None else None  # noqa: E731
    dx, dw = ops.rmsnorm_backward(view(dy), view(h), w.to(DEV) if w is not None else None, rstd.to(DEV), view(dh), need_dw,
                                  workspace)
    torch.cuda.synchronize()
    dx64, dw64, dx_size, dw_size = norm_bwd64(dy, h, w, rstd, dh)
    e = off(dx, dx64, rounding(dx64, h.dtype) + (norm_steps(cols) + 12) * U32 * dx_size)
    assert e <= 1, e
    if not need_dw:
        assert dw is None
        return e, 0.0
    f = off(dw, dw64, (rows + 8) * U32 * dw_size + 2.0 ** -149)
    assert f <= 1, f
    return e, f


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(700, 96), (1301, 640), (600, 2050), (70, 40000)])
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_norm_backward(rows, cols, t):
    g = gen(rows * 7919 + cols)
    h = torch.randn(rows, cols, generator=g).to(DT[t])
    dy = torch.randn(rows, cols, generator=g).to(DT[t])
    dh = torch.randn(rows, cols, generator=g).to(DT[t])
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(DT[t])
    _, rstd, _ = norm64(h, None, None, EPS)
    rstd = rstd.float()
    r = [check_bwd(dy, h, w, rstd, dh), check_bwd(dy, h, w.float(), rstd, None, pad=5, lead=1),
         check_bwd(dy, h, None, rstd, dh, workspace=None) if rows < 100 else (0, 0),
         check_bwd(dy, h, w, rstd, dh, workspace=torch.empty(5 * cols * 4, dtype=torch.uint8, device=DEV)),
         check_bwd(dy, h, w, rstd, dh, need_dw=False)]
    say(f"[norm backward] {t} {rows}x{cols}: dx {max(a for a, _ in r):.3f}, dw {max(b for _, b in r):.3f} of the tolerance")


def test_norm_backward_against_differences():
    """The gradient of sum(dy * y) + sum(dh * h) by central differences in 64 bits."""
    g = gen(3)
    rows, cols = 3, 37
    x, r = torch.randn(rows, cols, generator=g).double(), torch.randn(rows, cols, generator=g).double()
    x, r = x.float().double(), r.float().double()
    w = torch.randn(cols, generator=g).float().double()
    dy, dh = torch.randn(rows, cols, generator=g), torch.randn(rows, cols, generator=g)

    def f(x, w):
        h = x + r
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w
        return float((dy.double() * y).sum() + (dh.double() * h).sum())

    fwd = ops.rmsnorm(x.float().to(DEV), w.float().to(DEV), r.float().to(DEV))
    dx, dw = ops.rmsnorm_backward(dy.to(DEV), fwd.h, w.float().to(DEV), fwd.rstd, dh.to(DEV))
    step = 1e-5
    for i in range(rows):
        for j in range(0, cols, 5):
            d = torch.zeros_like(x)
            d[i, j] = step
            # the difference is off by step^2 and 64-bit noise / step, h by its rounding to fp32
            assert abs((f(x + d, w) - f(x - d, w)) / (2 * step) - float(dx[i, j])) < 2e-5
    for j in range(0, cols, 3):
        d = torch.zeros_like(w)
        d[j] = step
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * step) - float(dw[j])) < 2e-5


def test_norm_backward_of_no_rows_and_in_place():
    dw = torch.full((70,), 3.0, device=DEV)
    lg.check(lg.gemm_rmsnorm_bwd(lg.GEMM_BF16, 0, 0, 70, 0, 70, 0, 70, 0, 0, 0, 0, 0, 70, dw.data_ptr(), 0, 0,
                                 torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert bool((dw == 0).all())
    g = gen(9)
    for cols in (400, 5000, 40000):
        h, dy, dh = (torch.randn(12, cols, generator=g).bfloat16().to(DEV) for _ in range(3))
        rstd = torch.rand(12, generator=g).to(DEV) + 0.5
        want = ops.rmsnorm_backward(dy, h, None, rstd, dh)
        ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
        for place in (0, 1, 2):
            t = [dy.clone(), h.clone(), dh.clone()]
            got = torch.empty(cols, device=DEV)
            lg.check(lg.gemm_rmsnorm_bwd(lg.GEMM_BF16, 0, 12, cols, t[0].data_ptr(), cols, t[1].data_ptr(), cols, 0,
                                         rstd.data_ptr(), t[2].data_ptr(), cols, t[place].data_ptr(), cols, got.data_ptr(),
                                         ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))
            torch.cuda.synchronize()
            assert torch.equal(t[place], want[0]) and torch.equal(got, want[1])


# ------------------------------------------------------------------ products

def run_product(call, M, N, out, beta, pad, seed):
    """C = call(C's pointer, its type, its leading dimension) into rows `pad` apart; (C, its old values)."""
    old = torch.randn(M, N, generator=gen(seed)).to(out) if beta else torch.zeros(M, N, dtype=out)
    if not beta and M * N:
        old.view(torch.uint8).fill_(0xFF)   # NaN: must not be read
    C, whole = padded(old, pad, DEV)
    lg.check(call(C.data_ptr(), code(C), C.stride(0)))
    torch.cuda.synchronize()
    assert untouched(C, whole)
    return C.cpu(), old


def close(C, old, p64, size, steps, alpha, beta, cut=0.0):
    want = alpha * p64 + (beta * old.double() if beta else 0.0)
    allowed = rounding(want, C.dtype) + abs(alpha) * cut + U32 * (abs(alpha) * steps * size + 4 * want.abs()
                                               + (4 * abs(beta) * old.double().abs() if beta else 0.0))
    return off(C, want, allowed)


def stream():
    return torch.cuda.current_stream().cuda_stream


def f8_operands(M, N, K, seed):
    g = gen(seed)
    a, sa = ops.quantize_f8(torch.randn(M, K, generator=g))
    b, sb = ops.quantize_f8(torch.randn(N, K, generator=g))
    return a, sa, b, sb


WS = 16 << 20


def check_f8(M, N, K, out, alpha=1.0, beta=0.0, pads=(0, 0, 0), scales=True, ws=WS):
    a, sa, b, sb = f8_operands(M, N, K, M * 31 + N * 17 + K)
    if not scales:
        sa = sb = None
    A, B = padded(a, pads[0], DEV)[0], padded(b, pads[1], DEV)[0]
    SA, SB = (sa.to(DEV), sb.to(DEV)) if scales else (None, None)
    W = torch.full((max(ws, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    C, old = run_product(lambda c, t, ld: lg.gemm_f8(M, N, K, alpha, A.data_ptr(), A.stride(0), SA.data_ptr() if scales else 0,
                                                     B.data_ptr(), B.stride(0), SB.data_ptr() if scales else 0, beta, c, t, ld,
                                                     W.data_ptr() if ws else 0, ws, stream()), M, N, DT[out], beta, pads[2], K)
    p64, size = f8_64(a, b, sa, sb)
    cut = 0.0 if out == "f32" else f8_cut(a, b, sa, sb)
    e = close(C, old, p64, size, K + 4, alpha, beta, cut)   # K terms, three products by scales and alpha
    assert e <= 1, e
    return e


F8_SHAPES = [(1, 1, 1), (1, 5, 16), (3, 5, 15), (2, 17, 33), (16, 16, 128), (17, 33, 129), (64, 64, 255), (65, 70, 256),
             (1, 1000, 2048), (5, 321, 4100), (48, 257, 1024), (128, 128, 512), (130, 200, 2049), (256, 256, 256),
             (300, 520, 384), (257, 300, 1040), (512, 768, 640)]


@pytest.mark.parametrize("M,N,K", F8_SHAPES)
def test_f8(M, N, K):
    r = [check_f8(M, N, K, "f32"), check_f8(M, N, K, "bf16", ws=0), check_f8(M, N, K, "f16", 0.5, -1.5, (16, 32, 4)),
         check_f8(M, N, K, "f32", -2.0, 1.0, (1, 7, 3)), check_f8(M, N, K, "bf16", 1.0, 0.0, (0, 5, 1), scales=False),
         check_f8(M, N, K, "f32", 1.0, 0.0, (48, 16, 0), ws=4096)]
    say(f"[f8] {M}x{N}x{K}: {max(r):.3f} of the tolerance")


def test_f8_exact_integers():
    """Small whole numbers: every sum is exact, so every bit has to be right."""
    g = gen(1)
    for M, N, K in ((1, 96, 4096), (40, 33, 200), (256, 512, 1024)):
        a = torch.randint(-3, 4, (M, K), generator=g).float().to(torch.float8_e4m3fn)
        b = torch.randint(-3, 4, (N, K), generator=g).float().to(torch.float8_e4m3fn)
        C = ops.matmul_f8(a.to(DEV), b.to(DEV), out_dtype=torch.float32)
        assert torch.equal(C.cpu(), a.float() @ b.float().t())


@pytest.mark.parametrize("M,N,K,pad", [(4096, 4096, 512, 0), (4096, 4096, 128, 16), (4099, 4111, 650, 0), (4357, 3840, 255, 5),
                                       (2560, 12160, 384, 3), (640, 700, 8200, 0), (129, 260, 16000, 7)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_f8_exact_integers_large(M, N, K, pad, out):
    """The same on shapes that take the large tiles and the splits of K, from any pitch."""
    g = torch.Generator(DEV).manual_seed(M + K)
    draw = lambda rows: torch.randint(-3, 4, (rows, K), generator=g, device=DEV).float()  # noqa: E731
    a, b = draw(M), draw(N)
    A = padded(a.to(torch.float8_e4m3fn), pad, DEV)[0]
    B = padded(b.to(torch.float8_e4m3fn), pad, DEV)[0]
    want = a @ b.t()                                   # whole numbers below 2^24: exact in fp32
    C, whole = padded(torch.full((M, N), float("nan"), device=DEV).to(DT[out]), pad, DEV)
    ops.matmul_f8(A, B, C=C)
    assert untouched(C, whole)
    assert torch.equal(C, want.to(DT[out]))
    ops.matmul_f8(A, B, C=C, alpha=-2.0, beta=1.0, workspace=None)
    assert torch.equal(C, (-2.0 * want + want.to(DT[out]).float()).to(DT[out]))


def test_f8_nan_and_zero_stay_in_their_rows():
    M, N, K = 70, 90, 300
    a, sa, b, sb = f8_operands(M, N, K, 4)
    a[3, K - 1] = float("nan")
    b[7, 0] = float("nan")
    sa[5] = float("inf")
    a[9] = 0
    C = ops.matmul_f8(a.to(DEV), b.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=torch.float32).cpu()
    p64, size = f8_64(a, b, sa, sb)
    bad = torch.isnan(C)
    assert bool(bad[3].all()) and bool(bad[:, 7].all()) and int(bad.sum()) == M + N - 1
    fine = torch.ones(M, N, dtype=torch.bool)
    fine[3], fine[5], fine[:, 7] = False, False, False
    assert bool((C[9][torch.arange(N) != 7] == 0).all())
    assert float(((C.double() - p64).abs() / (U32 * (K + 4) * size + 2.0 ** -149))[fine].max()) <= 1
    assert bool(torch.isinf(C[5][torch.arange(N) != 7]).all())


def w4_operands(M, N, K, group, t, zeros, seed):
    g = gen(seed)
    a = torch.randn(M, K, generator=g).to(DT[t])
    codes, s, z = ops.quantize_w4(torch.randn(N, K, generator=g), group, DT[t], zeros)
    return a, codes, s, z


def check_w4(M, N, K, group, t, out, zeros, alpha=1.0, beta=0.0, pads=(0, 0, 0, 0), ws=WS):
    a, codes, s, z = w4_operands(M, N, K, group, t, zeros, M * 31 + N * 17 + K)
    A, Q = padded(a, pads[0], DEV)[0], padded(codes, pads[1], DEV)[0]
    S = padded(s, pads[2], DEV)[0]
    Z = padded(z, pads[2], DEV)[0] if zeros else None
    W = torch.full((max(ws, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    C, old = run_product(lambda c, ct, ld: lg.gemm_w4(code(A), M, N, K, group, alpha, A.data_ptr(), A.stride(0), Q.data_ptr(),
                                                      Q.stride(0), S.data_ptr(), Z.data_ptr() if zeros else 0, S.stride(0),
                                                      beta, c, ct, ld, W.data_ptr() if ws else 0, ws, stream()),
                         M, N, DT[out], beta, pads[3], K)
    p64, size = w4_64(a, codes, s, z, group)
    e = close(C, old, p64, size, min(group, K) + s.shape[1] + 16, alpha, beta)
    assert e <= 1, e
    return e


W4_SHAPES = [(1, 1, 1, 32), (1, 5, 31, 32), (2, 17, 33, 32), (3, 16, 64, 64), (1, 300, 1024, 128), (5, 70, 1000, 64),
             (16, 48, 2048, 128), (17, 33, 520, 32), (33, 100, 640, 96), (64, 65, 768, 256), (65, 130, 1025, 128),
             (128, 256, 512, 128), (200, 320, 1100, 64), (300, 257, 2048, 32), (256, 512, 1024, 1024)]


@pytest.mark.parametrize("M,N,K,group", W4_SHAPES)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_w4(M, N, K, group, t):
    r = [check_w4(M, N, K, group, t, t, False), check_w4(M, N, K, group, t, "f32", True, ws=0),
         check_w4(M, N, K, group, t, t, True, -0.5, 1.0, (8, 16, 0, 4)),
         check_w4(M, N, K, group, t, "f32", False, 2.0, -1.0, (1, 3, 1, 1)),
         check_w4(M, N, K, group, t, t, True, 1.0, 0.0, (0, 1, 5, 0), ws=4096)]
    say(f"[w4] {t} {M}x{N}x{K} by {group}: {max(r):.3f} of the tolerance")


@pytest.mark.parametrize("M,N,K,group,pad", [(2048, 2304, 1024, 128, 0), (2049, 2307, 1090, 64, 0), (1000, 1536, 640, 32, 3),
                                             (64, 1024, 8192, 128, 0), (100, 515, 8197, 64, 1), (300, 130, 16000, 32, 0),
                                             (257, 8200, 450, 192, 5), (33, 128, 64, 32, 0), (47, 200, 65, 64, 0),
                                             (4, 155, 14848, 128, 3), (3, 40, 5000, 96, 0), (2, 300, 20001, 64, 0),
                                             (1, 33, 40000, 32, 1), (1, 12400, 999, 128, 0), (4, 6300, 4097, 64, 0),
                                             (16, 155, 33000, 128, 0), (7, 4100, 9000, 32, 0), (20, 96, 20000, 64, 2)])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_w4_exact_integers_large(M, N, K, group, pad, t):
    """Small whole numbers: every sum is exact in fp32, so every bit has to be right, on the large tiles
    and the splits of K, from any pitch."""
    g = torch.Generator(DEV).manual_seed(M + K)
    groups = -(-K // group)
    a = torch.randint(-2, 3, (M, K), generator=g, device=DEV).float()
    codes = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = 2.0 ** torch.randint(-1, 2, (N, groups), generator=g, device=DEV).float()
    z = torch.randint(0, 16, (N, groups), generator=g, device=DEV).float()
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :K].float()
    each = lambda v: v.repeat_interleave(group, 1)[:, :K]  # noqa: E731
    A, Q = padded(a.to(DT[t]), pad, DEV)[0], padded(codes, pad, DEV)[0]
    S, Z = padded(s.to(DT[t]), pad, DEV)[0], padded(z.to(DT[t]), pad, DEV)[0]
    want = a @ (each(s) * (q - each(z))).t()
    C, whole = padded(torch.full((M, N), float("nan"), device=DEV), pad, DEV)
    ops.matmul_w4(A, Q, S, Z, group, C=C)
    assert untouched(C, whole)
    assert torch.equal(C, want)
    ops.matmul_w4(A, Q, S, None, group, C=C, alpha=-2.0, beta=1.0, workspace=torch.empty(1 << 16, dtype=torch.uint8, device=DEV))
    assert torch.equal(C, -2.0 * (a @ (each(s) * (q - 8.0)).t()) + want)
    low = ops.matmul_w4(A, Q, S, Z, group)
    assert torch.equal(low, want.to(DT[t]))


def test_w4_every_code_and_zero_point():
    """One element of A against every code and zero point: nothing is rounded before the end."""
    K = 32
    a = torch.zeros(2, K, dtype=torch.bfloat16)
    a[0, 5], a[1, 30] = 1.0, -2.0
    q = torch.arange(16, dtype=torch.uint8)
    q = (q | q << 4)[:, None].expand(16, K // 2)
    codes = q.repeat(16, 1).contiguous()                       # row 16 z + q: code q everywhere
    zeros = torch.arange(16).repeat_interleave(16)[:, None].to(torch.bfloat16)
    scales = torch.full((256, 1), 0.5, dtype=torch.bfloat16)
    C = ops.matmul_w4(a.to(DEV), codes.to(DEV), scales.to(DEV), zeros.to(DEV), group=32, out_dtype=torch.float32).cpu()
    want = 0.5 * (torch.arange(16).repeat(16) - zeros[:, 0].float())
    assert torch.equal(C, torch.stack([want, -2.0 * want]))


def test_w4_nan_stays_in_its_row_and_column():
    a, codes, s, _ = w4_operands(20, 50, 200, 64, "bf16", False, 8)
    a[3, 199] = float("nan")
    s[11, 2] = float("nan")
    a[4, 7] = float("inf")
    C = ops.matmul_w4(a.to(DEV), codes.to(DEV), s.to(DEV), group=64, out_dtype=torch.float32).cpu()
    bad = ~torch.isfinite(C)
    want = torch.zeros(20, 50, dtype=torch.bool)
    want[3], want[4], want[:, 11] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("alpha,K", [(0.0, 64), (1.0, 0)])
def test_products_that_only_scale_c(alpha, K):
    C0 = torch.randn(5, 7, device=DEV)
    for beta, want in ((0.0, torch.zeros_like(C0)), (-2.0, -2.0 * C0)):
        for op in ("f8", "w4"):
            C = C0.clone()
            if op == "f8":
                q = torch.zeros(8, K, dtype=torch.float8_e4m3fn, device=DEV)
                ops.matmul_f8(q[:5], q[:7], C=C, alpha=alpha, beta=beta)
            else:
                ops.matmul_w4(torch.zeros(5, K, dtype=torch.float16, device=DEV),
                              torch.zeros(7, K // 2, dtype=torch.uint8, device=DEV),
                              torch.ones(7, K // 32, dtype=torch.float16, device=DEV), group=32, C=C, alpha=alpha, beta=beta)
            assert torch.equal(C, want)


# ------------------------------------------------------------------ together

def chain(x, r, w, b, sb, codes, s, dy):
    n = ops.rmsnorm(x, w, r, out_dtype=torch.float8_e4m3fn)
    c = ops.matmul_f8(n.y, b, n.scale, sb)
    d = ops.matmul_w4(c, codes, s, group=64)
    dx, dw = ops.rmsnorm_backward(dy, n.h, w, n.rstd)
    return n.y.view(torch.uint8), n.scale, n.h, c, d, dx, dw


def chain_inputs(rows, seed):
    g = gen(seed)
    K, N = 512, 640
    x, r, dy = (torch.randn(rows, K, generator=g).bfloat16().to(DEV) for _ in range(3))
    w = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16().to(DEV)
    b, sb = ops.quantize_f8(torch.randn(N, K, generator=g))
    codes, s, _ = ops.quantize_w4(torch.randn(K, N, generator=g), 64, torch.bfloat16)
    return x, r, w, b.to(DEV), sb.to(DEV), codes.to(DEV), s.to(DEV), dy


@pytest.mark.parametrize("rows", [1, 33, 300])
def test_same_bits_again_and_on_another_stream(rows):
    args = chain_inputs(rows, rows)
    want = chain(*args)
    again = chain(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = chain(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, again, other):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("rows", [1, 65])
def test_graph_replays(rows):
    """Captured once, replayed with new inputs and eager work between: the eager results."""
    args = chain_inputs(rows, 1)
    chain(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(*args)
    for seed in (2, 3, 4):
        for t, v in zip(args, chain_inputs(rows, seed)):
            t.copy_(v)
        want = chain(*args)
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), seed


def test_example_block():
    """The example runs, and its block is as far from the unquantised one as 4-bit weights put it: a code is off by up
    to half a step of a fifteenth of its group's range, which for normal weights (groups of 128 span about 5 deviations)
    is 5 / 15 / sqrt(12) of one, a tenth, and the 8-bit rounding of y adds 2^-4 / sqrt(3) at most."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block.py")
    spec = importlib.util.spec_from_file_location("mlp_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off, out, dx, dw = example.main(["--width", "512", "--wide", "1024", "--prompt", "70", "--tokens", "3"])
    assert off < 0.15
    for t in (out, dx, dw):
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("M,N,K,pad", [(1, 20000, 512, 0), (5, 14000, 384, 16), (17, 6001, 640, 0), (29, 15003, 1040, 48),
                                       (32, 33000, 256, 0), (20, 9000, 1029, 3), (33, 700, 1024, 0), (47, 515, 4096, 16),
                                       (63, 9001, 256, 0)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_f8_few_rows_on_tiles(M, N, K, pad, out):
    """Fewer rows than a tile has, read without a copy of A: exact on small whole numbers, nothing written beside C."""
    g = torch.Generator(DEV).manual_seed(M + N + K)
    draw = lambda rows: torch.randint(-3, 4, (rows, K), generator=g, device=DEV).float()  # noqa: E731
    a, b = draw(M), draw(N)
    A = padded(a.to(torch.float8_e4m3fn), pad, DEV)[0]
    B = padded(b.to(torch.float8_e4m3fn), pad, DEV)[0]
    sa = 2.0 ** torch.randint(-1, 2, (M,), generator=g, device=DEV).float()
    sb = 2.0 ** torch.randint(-1, 2, (N,), generator=g, device=DEV).float()
    want = (a @ b.t()) * sa[:, None] * sb              # whole numbers by powers of two, below 2^24: exact in fp32
    C, whole = padded(torch.full((M, N), float("nan"), device=DEV).to(DT[out]), pad, DEV)
    for ws in ("auto", None):
        ops.matmul_f8(A, B, sa, sb, C=C, workspace=ws)
        assert untouched(C, whole)
        assert torch.equal(C, want.to(DT[out]))


@pytest.mark.parametrize("M,N,K,group,pad", [(33, 16384, 512, 128, 0), (40, 16500, 576, 64, 8), (63, 16384, 512, 32, 16),
                                             (48, 4096, 8192, 64, 0), (57, 4100, 9001, 64, 1)])
def test_w4_few_rows_on_tiles(M, N, K, group, pad):
    g = torch.Generator(DEV).manual_seed(M + N + K)
    groups = -(-K // group)
    a = torch.randint(-2, 3, (M, K), generator=g, device=DEV).float()
    codes = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = 2.0 ** torch.randint(-1, 2, (N, groups), generator=g, device=DEV).float()
    z = torch.randint(0, 16, (N, groups), generator=g, device=DEV).float()
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :K].float()
    each = lambda v: v.repeat_interleave(group, 1)[:, :K]  # noqa: E731
    A, Q = padded(a.bfloat16(), pad, DEV)[0], padded(codes, pad, DEV)[0]
    want = a @ (each(s) * (q - each(z))).t()
    C, whole = padded(torch.full((M, N), float("nan"), device=DEV), pad, DEV)
    ops.matmul_w4(A, Q, s.bfloat16(), z.bfloat16(), group, C=C)
    assert untouched(C, whole)
    assert torch.equal(C, want)


@pytest.mark.parametrize("group,t,zeros", [(32, "bf16", True), (64, "f16", True), (128, "bf16", True), (128, "f16", False)])
def test_w4_tiles_with_a_mean(group, t, zeros):
    """Rows of A with a large mean: what the zero points take off is many times what is left.  Zero points that are no
    whole numbers, scales of zero and of very different size."""
    M, N, K = 300, 4096, 2048
    a, codes, s, z = w4_operands(M, N, K, group, t, zeros, 77)
    a = (a.float() + 3.0).to(a.dtype)
    s[5] = 0.0
    s[9, ::2] = 2.0 ** -14
    if zeros:
        z = (z.float() + 0.37).to(z.dtype)
    C = ops.matmul_w4(a.to(DEV), codes.to(DEV), s.to(DEV), z.to(DEV) if zeros else None, group, out_dtype=torch.float32).cpu()
    p64, size = w4_64(a, codes, s, z, group)
    assert torch.equal(C[:, 5], torch.zeros(M))
    e = close(C, None, p64, size, group + s.shape[1] + 16, 1.0, 0.0)
    assert e <= 1, e


def test_w4_tiles_nan_stays_in_its_row_and_column():
    M, N, K, group = 300, 4096, 1000, 64
    a, codes, s, z = w4_operands(M, N, K, group, "bf16", True, 78)
    want = ops.matmul_w4(a.to(DEV), codes.to(DEV), s.to(DEV), z.to(DEV), group, out_dtype=torch.float32).cpu()
    a[17, K - 1], a[255, 3] = float("nan"), float("inf")
    s[4095, 0], z[40, s.shape[1] - 1] = float("nan"), float("inf")
    C = ops.matmul_w4(a.to(DEV), codes.to(DEV), s.to(DEV), z.to(DEV), group, out_dtype=torch.float32).cpu()
    rows = torch.ones(M, dtype=torch.bool)
    rows[[17, 255]] = False
    cols = torch.ones(N, dtype=torch.bool)
    cols[[40, 4095]] = False
    assert torch.equal(C[rows][:, cols], want[rows][:, cols])
    assert not C[~rows].isfinite().any() and not C[:, ~cols].isfinite().any()


@pytest.mark.parametrize("rows", [4, 5, 13, 16, 17, 40, 127, 128, 129])
@pytest.mark.parametrize("cols,t", [(4, "f32"), (37, "f32"), (250, "bf16"), (1000, "f16"), (3001, "f32"), (4097, "bf16"), (16000, "f16")])
def test_norm_backward_few_rows(rows, cols, t):
    """dw in the launch of dx: against the formula, every column once, and the bits of the two launches that a dx on dy takes."""
    g = gen(rows * 31 + cols)
    dy, h = (torch.randn(rows, cols, generator=g).to(DT[t]) for _ in range(2))
    w = torch.randn(cols, generator=g).to(DT[t])
    rstd = torch.rand(rows, generator=g) + 0.5
    DY, H = padded(dy, 3, DEV)[0], padded(h, 5, DEV)[0]
    W, R = w.to(DEV), rstd.to(DEV)
    ws = torch.empty(rows * cols * 4 + 256, dtype=torch.uint8, device=DEV)

    def run(a, dx):
        dw = torch.full((cols + 8,), float("nan"), device=DEV)
        lg.check(lg.gemm_rmsnorm_bwd(code(a), code(W), rows, cols, a.data_ptr(), a.stride(0), H.data_ptr(), H.stride(0),
                                     W.data_ptr(), R.data_ptr(), 0, 0, dx.data_ptr(), dx.stride(0), dw.data_ptr(),
                                     ws.data_ptr(), ws.numel(), stream()))
        torch.cuda.synchronize()
        assert bool(dw[cols:].isnan().all())
        return dx, dw[:cols]

    dx, dw = run(DY, torch.empty_like(DY))
    dx64, dw64, dx_size, dw_size = norm_bwd64(dy, h, w, rstd, None)
    assert off(dx, dx64, rounding(dx64, DT[t]) + (norm_steps(cols) + 12) * U32 * dx_size) <= 1
    assert off(dw, dw64, (rows + 8) * U32 * dw_size + 2.0 ** -149) <= 1
    mine = padded(dy, 3, DEV)[0]
    dx2, dw2 = run(mine, mine)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("M,lda", [(130, 4194368), (64, 4194368), (130, 8388608)])
def test_w4_rows_of_a_long_pitch(M, lda):
    """Rows of A that lie 8 MiB and more apart, below and past what the direct loads' offsets hold (128 rows of 2^24
    bytes): exact on small whole numbers."""
    N, K, group = 4096, 512, 64
    g = torch.Generator(DEV).manual_seed(lda + M)
    a = torch.randint(-2, 3, (M, K), generator=g, device=DEV).float()
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = 2.0 ** torch.randint(-1, 2, (N, K // group), generator=g, device=DEV).float()
    z = torch.randint(0, 16, (N, K // group), generator=g, device=DEV).float()
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1).float()
    each = lambda v: v.repeat_interleave(group, 1)  # noqa: E731
    A = torch.empty(M * lda, dtype=torch.bfloat16, device=DEV).view(M, lda)[:, :K]
    A.copy_(a)
    want = a @ (each(s) * (q - each(z))).t()
    C = ops.matmul_w4(A, codes, s.bfloat16(), z.bfloat16(), group, out_dtype=torch.float32)
    assert torch.equal(C, want)


@pytest.mark.parametrize("cols,t", [(2049, "bf16"), (2055, "bf16"), (4099, "bf16"), (1025, "f32"), (2051, "f16"), (9003, "bf16"), (4101, "f32")])
@pytest.mark.parametrize("rows", [3, 200])
def test_norm_backward_in_place_of_odd_widths(cols, t, rows):
    """dx on dy, on h and on dh where a row's last vector reaches into another wave's elements."""
    g = gen(cols)
    h, dy, dh = (torch.randn(rows, cols, generator=g).to(DT[t]).to(DEV) for _ in range(3))
    w = torch.randn(cols, generator=g).to(DT[t]).to(DEV)
    rstd = torch.rand(rows, generator=g).to(DEV) + 0.5
    want = ops.rmsnorm_backward(dy, h, w, rstd, dh)
    ws = torch.empty(rows * cols * 4 + 256, dtype=torch.uint8, device=DEV)
    for place in (0, 1, 2):
        a = [dy.clone(), h.clone(), dh.clone()]
        dw = torch.empty(cols, device=DEV)
        lg.check(lg.gemm_rmsnorm_bwd(code(h), code(h), rows, cols, a[0].data_ptr(), cols, a[1].data_ptr(), cols, w.data_ptr(),
                                     rstd.data_ptr(), a[2].data_ptr(), cols, a[place].data_ptr(), cols, dw.data_ptr(),
                                     ws.data_ptr(), ws.numel(), stream()))
        torch.cuda.synchronize()
        assert torch.equal(a[place], want[0]) and torch.equal(dw, want[1])


# ------------------------------------------------------------------ streams given by their handles

def each_call(rows=512):
    """(name, call(stream), the result that is kept) of every torch form that allocates."""
    x, r, w, b, sb, codes, s, dy = chain_inputs(rows, 11)
    n = ops.rmsnorm(x, w, r, out_dtype=torch.float8_e4m3fn)
    B = torch.randn(512, 640, generator=gen(4)).bfloat16().to(DEV)
    wide = torch.cat([x, r[:, :128]], 1)   # (here: what a call reads is there before its stream is chosen)
    return [("rmsnorm", lambda st: ops.rmsnorm(x, w, r, stream=st)[0]),
            ("rmsnorm to 8 bits", lambda st: ops.rmsnorm(x, w, r, out_dtype=torch.float8_e4m3fn, stream=st)[0].view(torch.uint8)),
            ("backward", lambda st: ops.rmsnorm_backward(dy, n.h, w, n.rstd, stream=st)[0]),
            ("f8", lambda st: ops.matmul_f8(n.y, b, n.scale, sb, stream=st)),
            ("w4", lambda st: ops.matmul_w4(wide, codes, s, group=64, stream=st)),
            ("bf16", lambda st: lg.matmul(x, B, stream=st, workspace="auto"))]


SPIN = 100_000_000   # of the device's clock: tens of milliseconds and more


@pytest.mark.parametrize("i", range(6))
def test_results_dropped_while_another_stream_writes_them(i):
    """What a call on a busy stream wrote and the caller dropped is not handed out before that stream is done."""
    name, call = each_call()[i]
    want = call(None).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sizes = [512 * 4, 512 * 4, 512 * 1024, 512 * 1280, 512 * 512, 640 * 4]   # rstd, scale, h or y, C, 8 bits, dw
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    call(side.cuda_stream)
    kept = call(side.cuda_stream)
    fresh = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes * 3]
    side.synchronize()
    torch.cuda.synchronize()
    for t in fresh:
        assert bool((t == 7).all()), name
    assert torch.equal(kept, want), name


@pytest.mark.parametrize("i", range(6))
def test_results_in_memory_that_the_current_stream_still_writes(i):
    """A call on another stream gets no block that was freed with work of the current stream still to come."""
    name, call = each_call()[i]
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty(want.numel() * want.element_size(), dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda._sleep(SPIN)
    for t in old:
        t.fill_(7)
    del old, t
    got = call(side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want), name


def test_inputs_dropped_while_another_stream_reads_them():
    x, r, w, b, sb, codes, s, dy = chain_inputs(512, 13)
    want = ops.matmul_w4(torch.cat([x, r[:, :128]], 1), codes, s, group=64)
    side = torch.cuda.Stream()
    wide = torch.cat([x, r[:, :128]], 1)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    size = wide.numel() * 2
    got = ops.matmul_w4(wide, codes, s, group=64, stream=side.cuda_stream)
    del wide
    fresh = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(bool((t == 7).all()) for t in fresh)


def test_the_default_stream_by_its_handle():
    x, r, w, b, sb, codes, s, dy = chain_inputs(33, 12)
    want = ops.rmsnorm(x, w, r)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = ops.rmsnorm(x, w, r, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got.y, want.y) and torch.equal(got.h, want.h)


@pytest.mark.parametrize("M,N,K,ws", [(1, 70, 640, WS), (20, 300, 200, WS), (40, 33, 90, 0), (64, 200, 512, WS), (200, 260, 384, 0),
                                      (129, 260, 8200, WS), (300, 520, 1000, WS), (512, 768, 640, WS)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_f8_scales_whose_product_leaves_the_range(M, N, K, ws, out):
    """Scales far from one whose results are ordinary floats: the product of two scales alone would be rounded to few bits,
    to 0 or to infinity.  A row of zeros with the largest scales stays one."""
    a, sa, b, sb = f8_operands(M, N, K, M + N + K)
    if M > 1:
        a[M // 2] = 0
    A, B = a.to(DEV), b.to(DEV)
    W = torch.empty(max(ws, 256), dtype=torch.uint8, device=DEV)
    for ea, eb in ((-66, -60), (-46, -80), (-100, -26), (110, -90), (-120, 60), (0, 0)):
        ta, tb = sa * 2.0 ** ea, sb * 2.0 ** eb
        tb[N // 3] = 2.0 ** 100
        if M > 1:
            ta[M // 2] = 2.0 ** 126
        C = ops.matmul_f8(A, B, ta.to(DEV), tb.to(DEV), out_dtype=DT[out], workspace=W if ws else None).cpu()
        p64, size = f8_64(a, b, ta, tb)
        cut = 0.0 if out == "f32" else f8_cut(a, b, ta.double(), tb.double())
        fine = p64.abs() < 2.0 ** 127
        e = off(torch.where(fine, C.double(), p64), p64, rounding(p64, DT[out]) + cut + U32 * ((K + 6) * size + 4 * p64.abs()))
        assert e <= 1, (ea, eb, e)
        assert int(fine.sum()) >= M * (N - 1) and (M == 1 or bool((C[M // 2] == 0).all()))


@pytest.mark.parametrize("M,N,K,group,ws", [(300, 4096, 4096, 128, "auto"), (300, 4096, 4096, 32, "auto"), (40, 16384, 4096, 64, "auto"),
                                            (200, 520, 8192, 192, "auto"), (256, 512, 8192, 32, "auto"), (300, 4096, 4095, 64, 8 << 20),
                                            (300, 4100, 4097, 32, 8 << 20), (300, 4096, 4095, 128, "auto"), (3, 200, 8192, 64, None),
                                            (16, 200, 8192, 128, None), (30, 200, 8191, 32, None)])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_w4_zero_points_come_off_group_by_group(M, N, K, group, ws, t):
    """Rows of A that are all positive: a * (1 + q/16) and a * (1 + z/16) add up to far more than 2^24 of their smallest parts
    over K, but in each group, and once the zero points are off, to less.  So an fp32 C that takes them off group by
    group is exact."""
    g = torch.Generator(DEV).manual_seed(M + N + K + group)
    groups = -(-K // group)
    a = torch.randint(200, 257, (M, K), generator=g, device=DEV)
    codes = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = 8.0 ** torch.randint(0, 2, (N, groups), generator=g, device=DEV).float()
    z = torch.randint(7, 10, (N, groups), generator=g, device=DEV).float()
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :K]
    each = lambda v: v.repeat_interleave(group, 1)[:, :K]  # noqa: E731
    w = (each(s) * (q.float() - each(z))).double()
    want = a.double() @ w.t()
    assert float(want.abs().max()) < 2 ** 24 and float((a.double()[:1] @ (each(s) * (16 + q.float())).double().t()).mean()) > 2 ** 26
    if isinstance(ws, int):
        ws = torch.empty(ws, dtype=torch.uint8, device=DEV)
    C = ops.matmul_w4(a.to(DT[t]), codes, s.to(DT[t]), z.to(DT[t]), group, out_dtype=torch.float32, workspace=ws)
    assert torch.equal(C.double(), want)


@pytest.mark.parametrize("M,N,K,op", [(2097120 + 2097152 + 17, 19, 32, "w4"), (5, (1 << 28) + 35, 1, "w4"), (2, (1 << 28) + 35, 1, "w4"),
                                      ((1 << 29) + 70, 1, 1, "f8"), (70, (1 << 24) + 35, 1, "f8"), (1, (1 << 28) + 35, 1, "f8")])
def test_sizes_beyond_one_launch(M, N, K, op):
    """More workgroups than a grid counts, without a workspace: exact on small whole numbers, the last rows and columns too."""
    g = torch.Generator(DEV).manual_seed(5)
    a = torch.randint(-2, 3, (M, K), generator=g, device=DEV, dtype=torch.int8)
    if op == "w4":
        codes = torch.randint(0, 16, (N, (K + 1) // 2), generator=g, device=DEV, dtype=torch.uint8) * 17   # both halves alike
        s = torch.ones(N, 1, dtype=torch.bfloat16, device=DEV)
        C = ops.matmul_w4(a.bfloat16(), codes, s, group=32, workspace=None)
        b = (codes & 15).to(torch.int8) - 8
        b = b.repeat_interleave(2, 1)[:, :K]
    else:
        b = torch.randint(-2, 3, (N, K), generator=g, device=DEV, dtype=torch.int8)
        sa = torch.full((M,), 2.0, device=DEV)
        sb = torch.ones(N, device=DEV)
        C = ops.matmul_f8(a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn), sa, sb, workspace=None)
        a = a * 2
    for m in range(0, M, 1 << 24):
        for n in range(0, N, 1 << 24):
            want = a[m:m + (1 << 24)].float() @ b[n:n + (1 << 24)].float().t()
            assert torch.equal(C[m:m + (1 << 24), n:n + (1 << 24)], want.bfloat16())


@pytest.mark.parametrize("cols", [40, 1000, 4096, 40000])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_norm_without_eps(cols, t):
    """eps = 0, or nearly, and rows whose squares leave fp32's range at either end: the norm is of the row as it stands."""
    g = gen(cols)
    x = torch.randn(12, cols, generator=g)
    x *= 2.0 ** torch.tensor([0, -40, -50, -62, -64, -75, -76, -100, -120, 62, 70, 110])[:, None]
    x = x.to(DT[t])
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(DT[t])
    for eps in (0.0, 2.0 ** -140, 2.0 ** -100):
        r = [check_norm(x, None, w, DT[out], eps=eps) for out in ("f32", "f8")]
        say(f"[norm without eps] {t} {cols} {eps}: {max(r):.3f} of the tolerance")


@pytest.mark.parametrize("rows,cols", [(400, 8192), (800, 4096), (300, 1000), (40, 40000), (3000, 7)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_norm_codes_are_the_quotients(rows, cols, t):
    """The 8-bit codes of a row are y / scale rounded once to fp32 and once to 8 bits, y as the call gives it in fp32.  Rows of
    few different values, where quotients lie on the border of two codes."""
    g = gen(rows + cols)
    x = torch.randn(rows, cols, generator=g).bfloat16()
    w = (1 + 0.1 * torch.randn(cols, generator=g)).bfloat16()
    x[::2] = (torch.randint(-40, 41, (rows, cols), generator=g) * 0.25).bfloat16()[::2]
    x, w = x.to(DT[t]).to(DEV), w.to(DT[t]).to(DEV)
    y = ops.rmsnorm(x, w, out_dtype=torch.float32)
    q = ops.rmsnorm(x, w, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(y.rstd, q.rstd)
    want = (y.y.cpu() / q.scale.cpu()[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q.y.cpu().view(torch.uint8), want.view(torch.uint8))


# ------------------------------------------------------------------ gradients through autograd

@pytest.mark.parametrize("rows,cols", [(1, 40), (7, 513), (300, 1000), (33, 4096)])
@pytest.mark.parametrize("t,wt,residual,used", [("f32", "f32", True, "both"), ("bf16", "bf16", True, "both"), ("f16", "f32", False, "both"),
                                                ("bf16", None, True, "y"), ("f32", "f32", True, "h"), ("bf16", "f32", False, "y")])
def test_norm_gradients_through_autograd(rows, cols, t, wt, residual, used):
    """backward() of a loss of y and h reaches x, residual and weight with what rmsnorm_backward gives, which is the formula's."""
    g = gen(rows + cols)
    draw = lambda dt: torch.randn(rows, cols, generator=g).to(dt).to(DEV)  # noqa: E731
    x, r = draw(DT[t]).requires_grad_(), draw(DT[t]).requires_grad_() if residual else None
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(DT[wt]).to(DEV).requires_grad_() if wt else None
    dy, dh = draw(DT[t]), draw(DT[t])
    n = ops.rmsnorm(x, w, r)
    with torch.no_grad():
        plain = ops.rmsnorm(x.detach(), w, r)
    assert torch.equal(n.y, plain.y) and torch.equal(n.h, plain.h) and torch.equal(n.rstd, plain.rstd)
    assert n.y.requires_grad and n.h.requires_grad and not n.rstd.requires_grad and not plain.y.requires_grad
    given = {"both": ([n.y, n.h], [dy, dh]), "y": ([n.y], [dy]), "h": ([n.h], [dh])}[used]
    torch.autograd.backward(*given)
    if used == "h":
        assert torch.equal(x.grad, dh) and torch.equal(r.grad, dh) and w.grad is None
        return
    up = dh if used == "both" else None
    dx, dw = ops.rmsnorm_backward(dy, plain.h, w.detach() if w is not None else None, plain.rstd,
                                  up if residual else None)
    if not residual and up is not None:
        dx = dx + up           # h is x itself: its gradient joins x's
    assert torch.equal(x.grad, dx)
    assert not residual or torch.equal(r.grad, dx)
    if w is not None:
        assert w.grad.dtype == w.dtype and torch.equal(w.grad, dw.to(w.dtype))
    dx64, dw64, dx_size, dw_size = norm_bwd64(dy.cpu(), plain.h.cpu(), w.detach().cpu() if w is not None else None,
                                              plain.rstd.cpu(), up.cpu() if up is not None else None)
    twice = 1 if residual else 2       # (roundings to x's type)
    assert off(x.grad, dx64, twice * rounding(dx_size, DT[t]) + (norm_steps(cols) + 12) * U32 * dx_size) <= 1
    if w is not None:
        assert off(w.grad, dw64, rounding(dw64, w.dtype) + (rows + 8) * U32 * dw_size + 2.0 ** -149) <= 1


def test_norm_gradients_of_another_output_type_and_of_strided_ones():
    """y in another type than x: its gradient comes in that type and is not rounded to x's; a gradient of no stride."""
    g = gen(3)
    rows, cols = 40, 1000
    x = torch.randn(rows, cols, generator=g).bfloat16().to(DEV).requires_grad_()
    w = torch.randn(cols, generator=g).bfloat16().to(DEV).requires_grad_()
    dy = torch.randn(rows, cols, generator=g).to(DEV)
    n = ops.rmsnorm(x, w, out_dtype=torch.float32)
    n.y.backward(dy)
    dx64, dw64, dx_size, dw_size = norm_bwd64(dy.cpu(), x.detach().cpu(), w.detach().cpu(), n.rstd.cpu(), None)
    assert off(x.grad, dx64, rounding(dx64, x.dtype) + (norm_steps(cols) + 12) * U32 * dx_size) <= 1
    assert off(w.grad, dw64, rounding(dw64, w.dtype) + (rows + 8) * U32 * dw_size) <= 1
    x.grad = None
    ops.rmsnorm(x, w).y.sum().backward()
    want, _ = ops.rmsnorm_backward(torch.ones_like(x), x.detach(), w.detach(), n.rstd)
    assert torch.equal(x.grad, want)
    x.grad = None
    wide = torch.randn(rows, 2 * cols, generator=g).bfloat16().to(DEV)
    (ops.rmsnorm(x, w).y.t() * wide[:, :cols].t()).sum().backward()
    want, _ = ops.rmsnorm_backward(wide[:, :cols].contiguous(), x.detach(), w.detach(), n.rstd)
    assert torch.equal(x.grad, want)


def test_gradients_that_there_are_not():
    """8-bit codes carry none, so a loss of them alone is refused; the products and second derivatives have none and say so."""
    g = gen(4)
    x = torch.randn(20, 64, generator=g).bfloat16().to(DEV).requires_grad_()
    r = torch.randn(20, 64, generator=g).bfloat16().to(DEV)
    n = ops.rmsnorm(x, None, r, out_dtype=torch.float8_e4m3fn)
    assert not n.y.requires_grad and not n.scale.requires_grad and n.h.requires_grad
    n.h.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))
    codes, s, _ = ops.quantize_w4(torch.randn(48, 64, generator=g), 32, torch.bfloat16)
    codes, s = codes.to(DEV), s.to(DEV)
    want = ops.matmul_w4(x.detach(), codes, s, group=32)
    C = torch.empty_like(want)
    for out in (None, C):
        got = ops.matmul_w4(x, codes, s, group=32, C=out)
        assert torch.equal(got, want) and (out is None or got.data_ptr() == C.data_ptr())
        with pytest.raises(RuntimeError, match="matmul_w4 has no backward pass"):
            got.sum().backward()
    q, sq = ops.quantize_f8(x.detach())
    got = ops.matmul_f8(q, q, sq.requires_grad_(), sq)
    with pytest.raises(RuntimeError, match="matmul_f8 has no backward pass"):
        got.sum().backward()
    with torch.no_grad():
        assert not ops.matmul_w4(x, codes, s, group=32).requires_grad
    dx, = torch.autograd.grad(ops.rmsnorm(x).y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_norm_gradients_on_another_stream():
    """The forward pass on a stream given by its handle, busy until later: the backward pass waits for it."""
    g = gen(6)
    x = torch.randn(300, 4096, generator=g).to(DEV).requires_grad_()
    r, dy = (torch.randn(300, 4096, generator=g).to(DEV) for _ in range(2))
    n = ops.rmsnorm(x, None, r)
    n.y.backward(dy)
    want, x.grad = x.grad, None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    y = ops.rmsnorm(x, None, r, stream=side.cuda_stream).y
    y.backward(dy)
    del y
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want)
