"""A transformer block's dense parts on the GPU against plain 64-bit forms: the product with bias, activation and residual, the
norm and rotation of heads, and their backward passes.  Tolerances are derived in block_util."""
import pytest
import torch

from block_util import ACTS, act64, heads64, heads_bwd64, linear64, linear_bwd64
from gpu_util import DEV, say
from ops_util import DT, off, padded, rounding, untouched
from tiled_stage_software_amd import libgemm as lg, ops

pytestmark = pytest.mark.gpu
EPS = 1e-6
CODE = {torch.float32: lg.GEMM_F32, torch.bfloat16: lg.GEMM_BF16, torch.float16: lg.GEMM_F16}
WS = 96 << 20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lg.load()  # fails loudly if the library is missing
    torch.zeros(1, device=DEV)


@pytest.fixture(scope="module")
def workspace():
    return torch.full((WS,), 0x7F, dtype=torch.uint8, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def stream():
    return torch.cuda.current_stream().cuda_stream


def at(t):
    return t.data_ptr() if t is not None else 0


# ------------------------------------------------------------------ product

def linear_inputs(M, N, K, t, out, seed, bias="in", residual=True):
    g = gen(seed)
    a = torch.randn(M, K, generator=g).to(DT[t])
    w = (torch.randn(N, K, generator=g) / max(K, 1) ** 0.5).to(DT[t])
    b = torch.randn(N, generator=g).to(DT[t] if bias == "in" else torch.float32) if bias else None
    r = torch.randn(M, N, generator=g).to(DT[out]) if residual else None
    return a, w, b, r


def run_linear(a, w, b, act, r, out, keep=True, pads=(0, 0, 0), lead=0, ws=None, in_place=False):
    """gemm_linear on rows pads (of a, w, the results) further apart; nothing else may be written."""
    M, K = a.shape
    N = w.shape[0]
    A, _ = padded(a, pads[0], DEV, lead=lead)
    W, _ = padded(w, pads[1], DEV, lead=lead)
    B = b.to(DEV) if b is not None else None
    C, Cw = padded(r if in_place else torch.zeros(M, N, dtype=DT[out]), pads[2], DEV, lead=lead)
    R = C if in_place else padded(r, pads[2], DEV, lead=lead)[0] if r is not None else None
    Z, Zw = padded(torch.zeros(M, N, dtype=a.dtype), pads[2], DEV, lead=lead)
    lg.check(lg.gemm_linear(CODE[a.dtype], M, N, K, at(A), A.stride(0), at(W), W.stride(0), at(B), CODE[b.dtype] if b is not None else 0,
                            ACTS.index(act), at(R), C.stride(0), at(Z) if keep else 0, Z.stride(0), at(C), CODE[DT[out]], C.stride(0),
                            at(ws), ws.numel() if ws is not None else 0, stream()))
    torch.cuda.synchronize()
    assert untouched(C, Cw) and untouched(Z, Zw)
    if not keep:
        assert bool((Z == 0).all())
    return C.cpu(), Z.cpu()


def check_linear(a, w, b, act, r, out, **kw):
    C, Z = run_linear(a, w, b, act, r, out, **kw)
    z, c, ez, ec = linear64(a, w, b, act, r)
    e = off(C, c, rounding(c, DT[out]) + ec)
    if kw.get("keep", True):
        e = max(e, off(Z, z, rounding(z, a.dtype) + ez))
    assert e <= 1, (act, out, kw, e)
    return e


LINEAR = [(1, 1, 1), (1, 64, 128), (3, 70, 40), (7, 129, 65), (16, 200, 512), (17, 96, 1000), (33, 300, 200), (64, 128, 640),
          (65, 257, 333), (130, 140, 64), (200, 513, 90), (257, 256, 448), (333, 401, 2049), (512, 768, 1024), (300, 520, 1000), (260, 300, 72), (1100, 2300, 264), (129, 131, 4101)]


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_linear(M, N, K, t, workspace):
    worst = 0.0
    for i, act in enumerate(ACTS):
        out = ("f32", t)[(i + M) % 2]
        a, w, b, r = linear_inputs(M, N, K, t, out, 7 * M + N + K + i, ("in", "f32", None)[(i + N) % 3], (i + K) % 3 != 0)
        pads = ((0, 0, 0), (8, 8, 8), (3, 1, 5))[i % 3]
        worst = max(worst, check_linear(a, w, b, act, r, out, keep=i % 2 == 0, pads=pads, lead=i % 2 * (i % 3 == 2),
                                        ws=workspace if i % 4 else None))
    say(f"[linear] {t} {M}x{N}x{K}: {worst:.3f} of the tolerance")


@pytest.mark.parametrize("M,N,K", [(5, 72, 100), (40, 264, 256), (300, 520, 192)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_residual_in_place(M, N, K, out, workspace):
    for pads in ((0, 0, 0), (0, 0, 3)):
        a, w, b, r = linear_inputs(M, N, K, "bf16", out, M + N)
        check_linear(a, w, b, "gelu", r, out, pads=pads, ws=workspace, in_place=True)


@pytest.mark.parametrize("act", ACTS)
def test_linear_of_no_depth(act):
    a, w, b, r = linear_inputs(5, 40, 0, "bf16", "f32", 3)
    check_linear(a, w, b, act, r, "f32")
    check_linear(a, w, None, act, None, "bf16")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_linear_activation_over_its_range(act, t):
    """Every finite value of the type (through an identity weight, in fp32), up to where exp2 leaves its range."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[t])
    v = bits[torch.isfinite(bits)]
    v = v[: len(v) // 64 * 64].view(-1, 64)
    v = v[(v.float().abs() < 2.0 ** 60).all(1)]
    eye = torch.eye(64, dtype=DT[t])
    C, Z = run_linear(v, eye, None, act, None, "f32")
    assert torch.equal(Z.float(), v.float())
    z, c, ez, ec = linear64(v, eye, None, act, None)
    e = off(C, c, rounding(c, torch.float32) + ec)
    say(f"[linear] {act} over {t}: {e:.3f} of the tolerance")
    assert e <= 1


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 20, 200])
def test_linear_nan_and_infinity_stay_in_their_rows(act, M, workspace):
    a, w, b, _ = linear_inputs(M, 96, 256, "bf16", "bf16", 5)
    a, w = a.abs(), w.abs()
    clean, _ = run_linear(a, w, b, act, None, "bf16", ws=workspace)
    a[1, 7] = float("nan")
    a[2, 200] = float("inf")
    C, Z = run_linear(a, w, b, act, None, "bf16", ws=workspace)
    assert bool(torch.isnan(C[1].float()).all()) and bool((C[2] == float("inf")).all())
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(C[keep], clean[keep])
    a[2, 200] = -float("inf")
    C, Z = run_linear(a, w, b, act, None, "bf16", ws=workspace)
    assert bool((Z[2] == -float("inf")).all())
    assert bool((C[2] == (-float("inf") if act == "none" else 0.0)).all())


def test_linear_exact_integers(workspace):
    """Small whole numbers are exact in every kernel, tile and split: 0/1 sums and a residual to the bit."""
    g = gen(8)
    for M, N, K in [(1, 256, 4096), (4, 100, 515), (16, 640, 1024), (31, 72, 900), (48, 200, 2048), (100, 128, 4096), (260, 300, 512),
                    (512, 512, 320)]:
        a = torch.randint(-2, 3, (M, K), generator=g).to(torch.bfloat16)
        w = torch.randint(-1, 2, (N, K), generator=g).to(torch.bfloat16)
        b = torch.randint(-8, 9, (N,), generator=g).float()
        r = torch.randint(-8, 9, (M, N), generator=g).float()
        want = torch.relu(a.double() @ w.double().t() + b.double()) + r.double()
        for ws in (workspace, None):
            C, _ = run_linear(a, w, b, "relu", r, "f32", ws=ws)
            assert torch.equal(C.double(), want), (M, N, K)


# ------------------------------------------------------------------ its backward pass

def check_linear_bwd(M, N, K, t, act, dc_type=None, dw_type=None, pads=(0, 0), ws=None, need=(True, True, True), on=None, seed=0):
    """on: what dZ lies on (None: memory of its own; "dc", "z")."""
    g = gen(seed + M + 3 * N + 5 * K)
    T, DC, DW = DT[t], DT[dc_type or t], DT[dw_type or t]
    dc = torch.randn(M, N, generator=g).to(DC)
    z = (1.5 * torch.randn(M, N, generator=g)).to(T) if act != "none" else None
    a = torch.randn(M, K, generator=g).to(T)
    w = (torch.randn(N, K, generator=g) / max(K, 1) ** 0.5).to(T)
    put = lambda v, pad: padded(v, pad, DEV)  # noqa: E731
    dC, A, W = put(dc, pads[0])[0], put(a, pads[1])[0], put(w, pads[1])[0]
    Z = put(z, pads[0])[0] if z is not None else None
    dZ, dZw = {"dc": (dC, None), "z": (Z, None)}.get(on) or put(torch.zeros(M, N, dtype=T), pads[0])
    dA, dAw = put(torch.zeros(M, K, dtype=T), pads[1])
    dW, dWw = put(torch.zeros(N, K, dtype=DW), pads[1])
    db = torch.full((N,), -7.0, device=DEV)
    null = act == "none" and DC == T and on is None
    lg.check(lg.gemm_linear_bwd(CODE[T], M, N, K, ACTS.index(act), at(dC), CODE[DC], dC.stride(0), at(Z), dC.stride(0), at(A), A.stride(0),
                                at(W), W.stride(0), 0 if null else at(dZ), dZ.stride(0), at(dA) if need[0] else 0, dA.stride(0),
                                at(dW) if need[1] else 0, CODE[DW], dW.stride(0), at(db) if need[2] else 0, at(ws),
                                ws.numel() if ws is not None else 0, stream()))
    torch.cuda.synchronize()
    assert untouched(dA, dAw) and untouched(dW, dWw) and (on or untouched(dZ, dZw))
    (dz64, da64, dw64, db64), (ez, ea, ew, eb) = linear_bwd64(dc, z, a, w, act, T)
    worst = 0.0
    if not null:
        worst = max(worst, off(dZ.cpu(), dz64, rounding(dz64, T) + ez))
    if need[0]:
        worst = max(worst, off(dA.cpu(), da64, rounding(da64, T) + ea))
    if need[1]:
        worst = max(worst, off(dW.cpu(), dw64, rounding(dw64, DW) + ew))
    if need[2]:
        worst = max(worst, off(db.cpu(), db64, rounding(db64, torch.float32) + eb))
    else:
        assert bool((db == -7.0).all())
    assert worst <= 1, (act, worst)
    return worst


LINEAR_BWD = [(1, 1, 1), (1, 64, 40), (5, 130, 72), (33, 40, 129), (64, 256, 200), (100, 300, 64), (257, 264, 256), (300, 513, 333),
              (513, 200, 643), (700, 520, 512)]


@pytest.mark.parametrize("M,N,K", LINEAR_BWD)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_linear_backward(M, N, K, t, workspace):
    worst = 0.0
    for i, act in enumerate(ACTS):
        worst = max(worst, check_linear_bwd(M, N, K, t, act, (None, "f32")[(i + M) % 2], (None, "f32")[(i + N) % 2],
                                            ((0, 0), (8, 8), (3, 5))[i % 3], workspace if i % 4 else None, seed=i,
                                            on=(None, "z", None, "dc", None)[i] if (i + M) % 2 == 0 else None))
    say(f"[linear backward] {t} {M}x{N}x{K}: {worst:.3f} of the tolerance")


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (False, False, False)])
def test_linear_backward_of_some(need, workspace):
    for act in ("none", "silu"):
        check_linear_bwd(70, 96, 88, "bf16", act, need=need, ws=workspace)


def test_linear_backward_of_no_rows(workspace):
    check_linear_bwd(0, 70, 40, "bf16", "gelu", ws=workspace)
    check_linear_bwd(4, 0, 40, "bf16", "none", ws=workspace)
    check_linear_bwd(4, 40, 0, "bf16", "relu", ws=workspace)


@pytest.mark.parametrize("act", ACTS)
def test_linear_slope_at_the_ends(act):
    """Infinities of Z (a rounded sum may be one) have the slope's limits, NaN stays."""
    z = torch.tensor([[float("inf"), -float("inf"), float("nan"), 3e38, -3e38, 100.0, -100.0, 0.0]], dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, 8, dtype=torch.bfloat16, device=DEV)
    _, _, db = ops.linear_backward(one, one[:, :1], torch.ones(8, 1, dtype=torch.bfloat16, device=DEV), z, act, (False, False, True))
    db = db.cpu()
    if act == "none":
        assert bool((db == 1).all())
        return
    assert torch.equal(db[[0, 3, 5]], torch.ones(3)) and bool((db[[1, 4, 6]].abs() < 1e-30).all()) and bool(torch.isnan(db[2]))
    assert float(db[7]) == pytest.approx(0.0 if act == "relu" else 0.5, abs=1e-6)


@pytest.mark.parametrize("act", ACTS[1:])
def test_linear_backward_against_differences(act):
    """d of sum(g * linear) along a direction, by central differences of the 64-bit form."""
    g = gen(17)
    a, w, b, _ = linear_inputs(24, 40, 56, "f16", "f32", 9, "f32", False)
    dy = torch.randn(24, 40, generator=g)
    y, z = ops.linear_keeping(a.to(DEV), w.to(DEV), b.to(DEV), act, out_dtype=torch.float32)
    dx, dw, db = ops.linear_backward(dy.to(DEV), a.to(DEV), w.to(DEV), z, act, dw_dtype=torch.float32)
    f = lambda a, w, b: float((dy.double() * act64(a @ w.t() + b, act)).sum())  # noqa: E731
    a, w, b = a.double(), w.double(), b.double()
    h = 1e-5
    for i, (v, got) in enumerate(((a, dx), (w, dw), (b, db))):
        d = torch.randn(v.shape, generator=g).double()
        args = [[a, w, b], [a, w, b]]
        args[0][i], args[1][i] = v + h * d, v - h * d
        want = (f(*args[0]) - f(*args[1])) / (2 * h)
        # each element of the gradients is off by a rounding of f16 or two (z's and dz's) of its terms: 2^-10 of their norms
        assert abs(float((got.double().cpu() * d).sum()) - want) <= 2.0 ** -10 * float(got.double().cpu().norm() * d.norm()) * 4


# ------------------------------------------------------------------ heads

def head_rows(v, dev_pad, order):
    """(device view of tokens x heads x dim, its whole buffer, the 2-D view in it): "tokens": token by token, heads side by side;
    "heads": head by head."""
    T, H, D = v.shape
    if order == "tokens":
        view, whole = padded(v.reshape(T, H * D), dev_pad, DEV)
        return view.unflatten(1, (H, D)), whole, view
    view, whole = padded(v.transpose(0, 1).reshape(H * T, D), dev_pad, DEV)
    return view.unflatten(0, (H, T)).transpose(0, 1), whole, view


def gh(t):
    return lg.GemmHeads(t.data_ptr(), t.stride(0), t.stride(1))


def heads_inputs(T, HQ, HK, D, rot, t, wt, seed, table=50):
    g = gen(seed)
    q, k = torch.randn(T, HQ, D, generator=g).to(DT[t]), (3 * torch.randn(T, HK, D, generator=g)).to(DT[t])
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(DT[wt]) if wt else None for _ in range(2)]
    pos = torch.randint(0, table, (T,), generator=g)
    angle = 6.3 * torch.rand(table, rot // 2, generator=g)
    return q, k, w, pos, (angle.cos(), angle.sin()) if rot else None


def rope_of(pos, angles, pairs):
    """(GemmRope or None, what it points to); the table's rows lie 3 floats further apart than they are long."""
    if angles is None:
        return None, None
    held = [padded(a, 3, DEV)[0] for a in angles] + [pos.to(DEV)]
    return lg.GemmRope(at(held[2]), at(held[0]), at(held[1]), held[0].stride(0), angles[0].shape[0], 2 * angles[0].shape[1],
                       ops.PAIRS[pairs]), held


def run_heads(q, k, w, pos, angles, pairs, pad=0, order="tokens", in_place=False, eps=EPS):
    T, HQ, D = q.shape
    (Q, Qw, Q2), (K, Kw, K2) = head_rows(q, pad, order), head_rows(k, pad, order)
    (OQ, OQw, OQ2), (OK, OKw, OK2) = ((Q, Qw, Q2), (K, Kw, K2)) if in_place else \
        (head_rows(torch.zeros_like(q), pad, order), head_rows(torch.zeros_like(k), pad, order))
    W = [v.to(DEV) if v is not None else None for v in w]
    rope, held = rope_of(pos, angles, pairs)
    lg.check(lg.gemm_qk_norm_rope(CODE[q.dtype], CODE[w[0].dtype] if w[0] is not None else 0, T, HQ, k.shape[1], D, eps, gh(Q), gh(K),
                                  at(W[0]), at(W[1]), rope, gh(OQ), gh(OK), stream()))
    torch.cuda.synchronize()
    assert untouched(OQ2, OQw) and untouched(OK2, OKw)
    return OQ.cpu(), OK.cpu()


def check_heads(q, k, w, pos, angles, pairs, **kw):
    worst = 0.0
    for got, x, wt in zip(run_heads(q, k, w, pos, angles, pairs, **kw), (q, k), w):
        y, e = heads64(x, wt, angles, pos, pairs, kw.get("eps", EPS))
        worst = max(worst, off(got, y, rounding(y, x.dtype) + e))
    assert worst <= 1, worst
    return worst


#         tokens, q heads, k heads, dim, rotated
HEADS = [(1, 1, 1, 1, 0), (1, 32, 8, 128, 128), (3, 4, 2, 64, 64), (5, 3, 1, 80, 40), (2, 2, 2, 128, 64), (4, 5, 5, 96, 96), (3, 1, 3, 72, 36),
         (2, 7, 1, 66, 2), (7, 2, 1, 33, 32), (3, 2, 1, 256, 256), (2, 3, 2, 250, 100), (2, 2, 1, 520, 520), (1, 1, 1, 1024, 512),
         (2, 1, 1, 1023, 1022), (70, 6, 2, 64, 32), (130, 3, 3, 16, 16), (9, 40, 8, 128, 128), (2, 65, 1, 112, 56), (4, 2, 1, 2, 2),
         (3, 2, 2, 192, 0)]


@pytest.mark.parametrize("T,HQ,HK,D,rot", HEADS)
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_heads(T, HQ, HK, D, rot, t):
    worst = 0.0
    for i, (pairs, wt, order, pad) in enumerate([("halves", t, "tokens", 0), ("neighbours", "f32", "tokens", 5), ("halves", None, "heads", 0),
                                                 ("neighbours", t, "heads", 3), ("halves", "f32", "tokens", 8)]):
        args = heads_inputs(T, HQ, HK, D, rot, t, wt, T + HQ + D + rot + i)
        worst = max(worst, check_heads(*args, pairs, pad=pad, order=order, in_place=i % 2 == 1))
    say(f"[heads] {t} {T}x({HQ}+{HK})x{D}, {rot} turned: {worst:.3f} of the tolerance")


def test_heads_of_one_kind_and_of_nothing():
    q, k, w, pos, angles = heads_inputs(5, 3, 2, 64, 64, "bf16", "bf16", 1)
    both = run_heads(q, k, w, pos, angles, "halves")
    rope, held = rope_of(pos, angles, "halves")
    for i, x in enumerate((q, k)):
        X, W = x.to(DEV), w[i].to(DEV)
        out = torch.empty_like(X)
        n = [x.shape[1] if i == j else 0 for j in range(2)]
        hs = [gh(X) if i == j else None for j in range(2)] + [gh(out) if i == j else None for j in range(2)]
        lg.check(lg.gemm_qk_norm_rope(lg.GEMM_BF16, lg.GEMM_BF16, 5, n[0], n[1], 64, EPS, hs[0], hs[1], at(W) if i == 0 else 0,
                                      at(W) if i == 1 else 0, rope, hs[2], hs[3], stream()))
        assert torch.equal(out.cpu(), both[i])
    out = ops.qk_norm_rope(q[:0].to(DEV), k[:0].to(DEV))
    assert out[0].shape == (0, 3, 64) and out[1].shape == (0, 2, 64)


@pytest.mark.parametrize("D,rot", [(64, 64), (80, 40), (128, 128), (256, 128)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_heads_special_rows(D, rot, pairs):
    """Zeros, NaN, infinities, the type's ends, and positions outside the table stay in their heads and tokens."""
    q, k, w, pos, angles = heads_inputs(6, 3, 3, D, rot, "bf16", "bf16", D)
    clean = run_heads(q, k, w, pos, angles, pairs)
    q2 = q.clone()
    q2[0, 1] = 0
    q2[1, 2, 5] = float("nan")
    q2[2, 0, D - 1] = float("inf")
    q2[3, 1] = 2.0 ** 100     # its square overflows
    q2[4, 1] = 2.0 ** -100    # its square vanishes beside eps
    got, kk = run_heads(q2, k, w, pos, angles, pairs)
    assert bool((got[0, 1] == 0).all()) and bool(torch.isnan(got[1, 2].float()).all())
    assert not bool(torch.isfinite(got[2, 0].float()).all())
    touched = {(0, 1), (1, 2), (2, 0), (3, 1), (4, 1)}
    for t in range(6):
        for h in range(3):
            if (t, h) not in touched:
                assert torch.equal(got[t, h], clean[0][t, h])
    assert torch.equal(kk, clean[1])
    check_heads(q2[3:5], k[3:5], w, pos[3:5], angles, pairs)
    for bad in (-1, 50, 1 << 40, -(1 << 62)):
        p2 = pos.clone()
        p2[2] = bad
        got = run_heads(q, k, w, p2, angles, pairs)
        for a, b in zip(got, clean):
            assert torch.equal(a[[0, 1, 3, 4, 5]], b[[0, 1, 3, 4, 5]])
            assert bool(torch.isnan(a[2, :, :rot].float()).all()) and torch.equal(a[2, :, rot:], b[2, :, rot:])


def test_heads_without_eps():
    q, k, w, pos, angles = heads_inputs(4, 2, 2, 128, 128, "f32", "f32", 2)
    for by in (2.0 ** -70, 1.0, 2.0 ** 70):
        check_heads(q * by, k * by, w, pos, angles, "halves", eps=0.0)


def check_heads_bwd(q, k, w, pos, angles, pairs, pad=0, order="tokens", on=None, ws=None, need_dw=True, eps=EPS):
    T, HQ, D = q.shape
    g = gen(T + D)
    dq, dk = torch.randn(q.shape, generator=g).to(q.dtype), torch.randn(k.shape, generator=g).to(q.dtype)
    Q, K, DQ, DK = (head_rows(v, pad, order) for v in (q, k, dq, dk))
    OQ, OK = {"x": (Q, K), "dy": (DQ, DK)}.get(on) or (head_rows(torch.zeros_like(q), pad, order), head_rows(torch.zeros_like(k), pad, order))
    W = [v.to(DEV) if v is not None else None for v in w]
    dw = torch.full((2, D), -7.0, device=DEV)
    rope, held = rope_of(pos, angles, pairs)
    lg.check(lg.gemm_qk_norm_rope_bwd(CODE[q.dtype], CODE[w[0].dtype] if w[0] is not None else 0, T, HQ, k.shape[1], D, eps, gh(DQ[0]),
                                      gh(DK[0]), gh(Q[0]), gh(K[0]), at(W[0]), at(W[1]), rope, gh(OQ[0]), gh(OK[0]),
                                      at(dw[0]) if need_dw else 0, at(dw[1]) if need_dw else 0, at(ws), ws.numel() if ws is not None else 0,
                                      stream()))
    torch.cuda.synchronize()
    assert untouched(OQ[2], OQ[1]) and untouched(OK[2], OK[1])
    worst = 0.0
    for i, (x, dy, got) in enumerate(((q, dq, OQ[0]), (k, dk, OK[0]))):
        (dx64, dw64), (ex, ew) = heads_bwd64(dy, x, w[i], angles, pos, pairs, eps)
        worst = max(worst, off(got.cpu(), dx64, rounding(dx64, x.dtype) + ex))
        if need_dw:
            worst = max(worst, off(dw[i].cpu(), dw64, rounding(dw64, torch.float32) + ew))
    if not need_dw:
        assert bool((dw == -7.0).all())
    assert worst <= 1, worst
    return worst


@pytest.mark.parametrize("T,HQ,HK,D,rot", HEADS)
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_heads_backward(T, HQ, HK, D, rot, t, workspace):
    worst = 0.0
    for i, (pairs, wt, order, pad) in enumerate([("halves", t, "tokens", 0), ("neighbours", "f32", "tokens", 5), ("halves", None, "heads", 0),
                                                 ("neighbours", t, "heads", 3), ("halves", "f32", "tokens", 8)]):
        args = heads_inputs(T, HQ, HK, D, rot, t, wt, T + HQ + D + rot + i)
        worst = max(worst, check_heads_bwd(*args, pairs, pad=pad, order=order, on=(None, "x", "dy", None, None)[i],
                                           ws=(workspace, None, workspace, workspace[:4096 * D], workspace)[i], need_dw=i != 4))
    say(f"[heads backward] {t} {T}x({HQ}+{HK})x{D}, {rot} turned: {worst:.3f} of the tolerance")


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_heads_backward_of_many_tokens(t, workspace):
    """Many parts of dw, and the same bits again."""
    args = heads_inputs(3001, 6, 2, 64, 64, t, t, 4)
    say(f"[heads backward] {check_heads_bwd(*args, 'halves', ws=workspace):.3f}")


def test_heads_backward_of_nothing():
    z = torch.zeros(0, 3, 64, device=DEV)
    out = ops.qk_norm_rope_backward(z, z[:, :1], z, z[:, :1], torch.ones(64, device=DEV), torch.ones(64, device=DEV))
    assert bool((out[2] == 0).all()) and bool((out[3] == 0).all()) and out[0].shape == (0, 3, 64)


def test_heads_backward_against_differences():
    g = gen(21)
    q, k, w, pos, angles = heads_inputs(6, 3, 2, 32, 16, "f32", "f32", 5)
    dq, dk = torch.randn(q.shape, generator=g), torch.randn(k.shape, generator=g)
    cos, sin = (a.to(DEV) for a in angles)
    for pairs in ops.PAIRS:
        got = ops.qk_norm_rope_backward(*(t.to(DEV) for t in (dq, dk, q, k, *w, pos)), cos, sin, pairs, EPS)
        f = lambda q, k, a, b: float((dq.double() * heads64(q, a, angles, pos, pairs, EPS)[0]).sum() +  # noqa: E731
                                     (dk.double() * heads64(k, b, angles, pos, pairs, EPS)[0]).sum())
        args = [t.double() for t in (q, k, *w)]
        for i in range(4):
            d = torch.randn(args[i].shape, generator=g).double()
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
            want = (f(*up) - f(*down)) / 2e-5
            assert abs(float((got[i].double().cpu() * d).sum()) - want) <= 1e-5 * float(got[i].double().cpu().norm() * d.norm())
