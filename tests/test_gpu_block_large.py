"""The large tiles of the product with bias, activation and residual and of its backward pass, on sizes that they do not divide:
rows, columns and depth that end inside a tile or a slab, each way of loading, each type of result.

The 64-bit forms are those of block_util, on the GPU for their size."""
import pytest
import torch

from block_util import SLOPE, act64, act_error, slope64
from gpu_util import DEV, say
from ops_util import DT, U32, padded, rounding, untouched
from test_gpu_block import ACTS, CODE, at, gen, run_linear, stream
from tiled_stage_software_amd import libgemm as lg

pytestmark = pytest.mark.gpu
WS = 512 << 20

# Rows, columns, depth of products that tiles of 256 x 256 and of 192 x 256 take (test_block_plans_cpu holds them to it): whole slabs
# and a part of one, one slab and several, edges in each direction.
LINEAR_256 = [(4001, 4090, 328), (4096, 4096, 64), (4096, 3900, 1000)]
LINEAR_192 = [(2600, 4600, 328), (1536, 8192, 72), (2477, 4603, 640)]
# Rows, N, K of backward passes: dA on 256 x 256, dW on them, both.
GRAD_A, GRAD_W, GRAD_BOTH = [(4001, 328, 4090), (4000, 72, 4096)], [(328, 4001, 4090), (72, 4000, 4096)], [(4096, 4090, 4001)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lg.load()  # fails loudly if the library is missing
    torch.zeros(1, device=DEV)


@pytest.fixture(scope="module")
def workspace():
    ws = torch.full((WS,), 0x7F, dtype=torch.uint8, device=DEV)
    yield ws
    del ws
    torch.cuda.empty_cache()


def worst(got, want, allowed):
    """The largest error over what is allowed, on the GPU (all finite)."""
    got = got.to(DEV).double()
    assert bool(torch.isfinite(got).all())
    return float(((got - want).abs() / allowed).max())


def check(a, w, b, act, r, out, **kw):
    C, Z = run_linear(a, w, b, act, r, out, **kw)
    again = run_linear(a, w, b, act, r, out, **kw)
    assert torch.equal(C, again[0]) and torch.equal(Z, again[1])
    a, w = a.to(DEV).double(), w.to(DEV).double()
    z, size = a @ w.t(), a.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b.to(DEV).double(), size + b.to(DEV).double().abs()
    ez = (a.shape[1] + 6) * U32 * size                  # (a rounding of the terms' magnitudes each, bias and joins)
    c = act64(z, act)
    ec = 1.13 * ez + act_error(z, act)                  # (no activation is steeper than 1.13)
    if r is not None:
        ec = ec + 2 * U32 * (c.abs() + r.to(DEV).double().abs())
        c = c + r.to(DEV).double()
    e = worst(C, c, rounding(c, DT[out]) + ec)
    if kw.get("keep", True):
        e = max(e, worst(Z, z, rounding(z, Z.dtype) + ez))
    return e


@pytest.mark.parametrize("M,N,K", LINEAR_256 + LINEAR_192)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_linear_on_large_tiles(M, N, K, t, workspace):
    g = gen(M + N + K)
    a = torch.randn(M, K, generator=g).to(DT[t])
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(DT[t])
    b = torch.randn(N, generator=g)
    r = torch.randn(M, N, generator=g)
    e = 0.0
    for i, (act, out, pads, ws, in_place) in enumerate([("gelu", t, (0, 0, 0), None, True), ("silu", "f32", (8, 8, 8), workspace, False),
                                                        ("gelu_tanh", t, (3, 1, 5), workspace, False), ("none", "f32", (0, 0, 1), None, False)]):
        e = max(e, check(a, w, (b if i % 2 else b.to(DT[t])) if i != 3 else None, act, r.to(DT[out]) if i != 2 else None, out, keep=i != 1,
                         pads=pads, ws=ws, in_place=in_place))
    say(f"[linear, large tiles] {t} {M}x{N}x{K}: {e:.3f} of the tolerance")
    assert e <= 1


@pytest.mark.parametrize("M,N,K", LINEAR_256 + LINEAR_192)
def test_linear_exact_integers_on_large_tiles(M, N, K, workspace):
    """Sums of small whole numbers are exact in any order: to the bit, in rows of any alignment."""
    g = gen(8)
    a = torch.randint(-2, 3, (M, K), generator=g).to(torch.bfloat16)
    w = torch.randint(-1, 2, (N, K), generator=g).to(torch.bfloat16)
    b = torch.randint(-8, 9, (N,), generator=g).float()
    r = torch.randint(-8, 9, (M, N), generator=g).float()
    z = a.to(DEV).double() @ w.to(DEV).double().t() + b.to(DEV).double()
    for pads, ws in (((0, 0, 0), None), ((8, 8, 0), None), ((1, 3, 5), workspace)):
        C, Z = run_linear(a, w, b, "relu", r, "f32", pads=pads, ws=ws)
        assert torch.equal(C.to(DEV).double(), torch.relu(z) + r.to(DEV).double()), pads
        assert torch.equal(Z.to(DEV), z.to(torch.bfloat16)), pads


def run_backward(dc, z, a, w, act, dw_type, pads, ws):
    """(dZ, dA, dW, db) of gemm_linear_bwd on rows pads (of M x N, of the others) further apart."""
    M, K = a.shape
    N, T = w.shape[0], a.dtype
    dC, A, W = padded(dc, pads[0], DEV)[0], padded(a, pads[1], DEV)[0], padded(w, pads[1], DEV)[0]
    Z = padded(z, pads[0], DEV)[0] if act != "none" else None
    dZ, dZw = padded(torch.zeros(M, N, dtype=T), pads[0], DEV)
    dA, dAw = padded(torch.zeros(M, K, dtype=T), pads[1], DEV)
    dW, dWw = padded(torch.zeros(N, K, dtype=DT[dw_type]), pads[1], DEV)
    db = torch.full((N,), -7.0, device=DEV)
    lg.check(lg.gemm_linear_bwd(CODE[T], M, N, K, ACTS.index(act), at(dC), CODE[dc.dtype], dC.stride(0), at(Z), dC.stride(0), at(A), A.stride(0),
                                at(W), W.stride(0), at(dZ), dZ.stride(0), at(dA), dA.stride(0), at(dW), CODE[DT[dw_type]], dW.stride(0), at(db),
                                at(ws), ws.numel() if ws is not None else 0, stream()))
    torch.cuda.synchronize()
    assert untouched(dA, dAw) and untouched(dW, dWw) and untouched(dZ, dZw)
    return tuple(t.clone() for t in (dZ, dA, dW, db))


@pytest.mark.parametrize("M,N,K", GRAD_A + GRAD_W + GRAD_BOTH)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_linear_backward_on_large_tiles(M, N, K, t, workspace):
    T = DT[t]
    g = gen(M + 3 * N + 5 * K)
    dc, z = torch.randn(M, N, generator=g), (1.5 * torch.randn(M, N, generator=g)).to(T)
    a = torch.randn(M, K, generator=g).to(T)
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(T)
    A, W = a.to(DEV).double(), w.to(DEV).double()
    e = 0.0
    for act, dc_type, dw_type, pads, ws in [("gelu", t, t, (0, 0), workspace), ("silu", "f32", "f32", (8, 8), None), ("none", t, "f32", (3, 5), workspace)]:
        dC = dc.to(DT[dc_type])
        got = run_backward(dC, z, a, w, act, dw_type, pads, ws)
        if ws is not None:
            ws.fill_(0x3C)
        for x, y in zip(got, run_backward(dC, z, a, w, act, dw_type, pads, ws)):
            assert torch.equal(x, y)                                        # (whatever the workspace holds)
        d = dC.to(DEV).double()
        dz = d if act == "none" else d * slope64(z.to(DEV).double(), act)
        e0 = d.abs() * (SLOPE if act != "none" else 0.0) + U32 * dz.abs()    # (as linear_bwd64 has it)
        ez = e0 + rounding(dz, T)
        mag = dz.abs() + ez
        e = max(e, worst(got[0], dz, rounding(dz, T) + e0))
        da, dw, db = dz @ W, dz.t() @ A, dz.sum(0)
        e = max(e, worst(got[1], da, rounding(da, T) + ez @ W.abs() + (N + 6) * U32 * (mag @ W.abs())))
        e = max(e, worst(got[2], dw, rounding(dw, DT[dw_type]) + ez.t() @ A.abs() + (M + 6) * U32 * (mag.t() @ A.abs())))
        e = max(e, worst(got[3], db, rounding(db, torch.float32) + e0.sum(0) + (M + 6) * U32 * mag.sum(0)))
    say(f"[linear backward, large tiles] {t} {M}x{N}x{K}: {e:.3f} of the tolerance")
    assert e <= 1


@pytest.mark.parametrize("M,N,K", GRAD_A + GRAD_W + GRAD_BOTH)
@pytest.mark.parametrize("dw_type", ["bf16", "f32"])
def test_linear_backward_exact_integers_on_large_tiles(M, N, K, dw_type, workspace):
    """Small whole numbers: the sums are exact, and a 16-bit result is their one rounding."""
    g = gen(9)
    ints = lambda n, *s: torch.randint(-n, n + 1, s, generator=g).to(torch.bfloat16)  # noqa: E731
    dc, z, a, w = ints(2, M, N), ints(3, M, N), ints(2, M, K), ints(1, N, K)
    dz = (dc.to(DEV).double() * (z.to(DEV) > 0)).double()
    da, dw = dz @ w.to(DEV).double(), dz.t() @ a.to(DEV).double()
    for pads, ws in (((0, 0), None), ((8, 8), workspace), ((1, 3), workspace)):
        got = run_backward(dc, z, a, w, "relu", dw_type, pads, ws)
        assert torch.equal(got[0].double(), dz) and torch.equal(got[3].double(), dz.sum(0)), pads
        assert torch.equal(got[1], da.to(torch.bfloat16)) and torch.equal(got[2], dw.to(DT[dw_type])), pads


@pytest.mark.parametrize("M,N,K", [(300, 513, 333), (513, 1001, 643), GRAD_A[0], GRAD_W[0], GRAD_BOTH[0]])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_backward_rounds_dz_once_and_nothing_else(M, N, K, t, workspace):
    """The one rounding to 16 bits inside the backward pass is dZ's: dA and dW are the products of the dZ that is stored, to fp32
    sums and their own rounding, and db is the sum of the unrounded values."""
    T = DT[t]
    g = gen(M + N + K)
    dc, z = torch.randn(M, N, generator=g).to(T), (1.5 * torch.randn(M, N, generator=g)).to(T)
    a, w = torch.randn(M, K, generator=g).to(T), (torch.randn(N, K, generator=g) / K ** 0.5).to(T)
    dZ, dA, dW, db = run_backward(dc, z, a, w, "gelu", "f32", (0, 0), workspace)
    A, W, dz = a.to(DEV).double(), w.to(DEV).double(), dc.to(DEV).double() * slope64(z.to(DEV).double(), "gelu")
    kept, slope = dZ.double(), dc.to(DEV).double().abs() * SLOPE + U32 * dz.abs()
    assert worst(dZ, dz, rounding(dz, T) + slope) <= 1
    da, dw = kept @ W, kept.t() @ A
    assert worst(dA, da, rounding(da, T) + (N + 6) * U32 * (kept.abs() @ W.abs())) <= 1
    assert worst(dW, dw, rounding(dw, torch.float32) + (M + 6) * U32 * (kept.abs().t() @ A.abs())) <= 1
    far = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
    say(f"[linear backward] {t} {M}x{N}x{K}: dA {far(dA, dz @ W):.1e}, dW (fp32) {far(dW, dz.t() @ A):.1e}, db {far(db, dz.sum(0)):.1e} "
        f"from 64 bits; from the products of the rounded dZ {far(dA, da):.1e}, {far(dW, dw):.1e}")
    assert worst(db, dz.sum(0), rounding(dz.sum(0), torch.float32) + slope.sum(0) + (M + 6) * U32 * (dz.abs() + slope).sum(0)) <= 1
