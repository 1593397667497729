"""Ends of a transformer block's dense parts on the GPU: infinite weights where the depth ends inside a slab, far tails of the
activations, the same bits from many parts."""
import math

import pytest
import torch

from block_util import ACTS, act64
from gpu_util import DEV, say
from test_gpu_block import EPS, gen, heads_inputs, run_linear
from test_gpu_block_large import run_backward
from tiled_stage_software_amd import libgemm as lg, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lg.load()  # fails loudly if the library is missing
    torch.zeros(1, device=DEV)


@pytest.fixture(scope="module")
def workspace():
    return torch.full((96 << 20,), 0x7F, dtype=torch.uint8, device=DEV)


#          few rows (one to four, a block, two blocks; eight waves and sixteen), tiles of 64 and of 128 rows, depths below a slab
INFINITE = [(3, 70, 72), (3, 70, 2049), (13, 96, 72), (13, 96, 1100), (20, 96, 72), (20, 96, 2049), (20, 9000, 130), (40, 96, 72),
            (64, 300, 1000), (200, 260, 72), (333, 401, 2049), (260, 300, 129), (200, 96, 40)]


@pytest.mark.parametrize("M,N,K", INFINITE)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_infinite_weights_reach_their_columns_alone(M, N, K, t, workspace):
    """Elements that a last slab reads for the second time count once: an infinite weight among them makes its column's sums
    infinite (not NaN), a NaN makes them NaN, and the other columns keep their bits."""
    dtype = torch.bfloat16 if t == "bf16" else torch.float16
    g = gen(M + N + K)
    a = (torch.rand(M, K, generator=g) + 0.1).to(dtype)
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(dtype)
    inf = float("inf")
    odd = {5: (max(K // 64 * 64 - 1, 0), inf), 6: (max(K - 64, 0), -inf), 17: (max(K - 60, 0), float("nan")), 33: (K - 1, inf), 34: (0, -inf)}
    v = w.clone()
    for n, (k, x) in odd.items():
        v[n, k] = x
    keep = [n for n in range(N) if n not in odd]
    for pad in (0, 8, 3):
        for ws in (workspace, None):
            for act in ("none", "silu"):
                clean, clean_z = run_linear(a, w, None, act, None, t, pads=(pad, pad, 0), ws=ws)
                C, Z = run_linear(a, v, None, act, None, t, pads=(pad, pad, 0), ws=ws)
                assert torch.equal(C[:, keep], clean[:, keep]) and torch.equal(Z[:, keep], clean_z[:, keep])
                for n, (k, x) in odd.items():
                    if x != x:
                        assert bool(torch.isnan(C[:, n].float()).all() and torch.isnan(Z[:, n].float()).all()), (n, pad, act, ws is None)
                    else:
                        limit = x if act == "none" or x > 0 else 0.0
                        assert bool((Z[:, n] == x).all() and (C[:, n] == limit).all()), (n, pad, act, ws is None)


@pytest.mark.parametrize("act", ACTS[2:])
def test_activations_keep_their_bound_in_far_tails(act):
    """Any fp32 sum (a bias on sums of zeros): 2^-20 + q 2^-22 of the value, or 2^-119 where exp2 has underflown, and the roundings of C
    and of the last sum."""
    b = torch.cat([torch.linspace(-140, 20, 40000), torch.linspace(-15, -5, 20000), torch.tensor([-1e4, -3e4, -1e30, 1e30])])
    b = torch.nn.functional.pad(b, (0, -len(b) % 64))
    a, w = torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(len(b), 64, dtype=torch.bfloat16)
    C, _ = run_linear(a, w, b, act, None, "f32", keep=False)
    z = b.double()
    q = {"gelu": z * z / 2, "gelu_tanh": math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3).abs(), "silu": z.abs()}[act]
    want = act64(z, act)
    e = ((C[0].double() - want).abs() / ((want.abs() * (2.0 ** -20 + q * 2.0 ** -22 + 2.0 ** -24)).clamp_min(2.0 ** -119))).max()
    say(f"[linear] {act} to its tail: {float(e):.3f} of the bound")
    assert float(e) <= 1


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("T,HQ,HK,D,rot", [(3001, 6, 2, 64, 64), (513, 5, 1, 72, 36), (2049, 3, 3, 40, 10)])
def test_heads_backward_gives_the_same_bits_again(T, HQ, HK, D, rot, t, workspace):
    """Many parts of dw: in the same order whatever the workspace holds."""
    q, k, w, pos, angles = heads_inputs(T, HQ, HK, D, rot, t, t, 4)
    g = gen(T)
    dq, dk = (torch.randn(x.shape, generator=g).to(x.dtype) for x in (q, k))
    args = [x.to(DEV) for x in (dq, dk, q, k, *w, pos, *angles)]
    runs = []
    for fill in (0x7F, 0x00, 0x3C):
        workspace.fill_(fill)
        runs.append(ops.qk_norm_rope_backward(*args, eps=EPS, workspace=workspace))
    for again in runs[1:]:
        for x, y in zip(runs[0], again):
            assert torch.equal(x, y)
    assert lg.gemm_qk_norm_rope_bwd_workspace_size(lg.GEMM_F32, T, HQ, HK, D)[1] > 64 * D * 4


@pytest.mark.parametrize("M,N,K", [(70, 96, 88), (33, 40, 129), (300, 513, 333), (513, 200, 643), (4001, 328, 4090)])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_infinite_operands_of_the_backward_pass_reach_their_columns_alone(M, N, K, t, workspace):
    """An infinity in W or A reaches its column of dA or dW, a NaN in dC its row of dA and of dW: wherever sums end inside a slab."""
    dtype = torch.bfloat16 if t == "bf16" else torch.float16
    g = gen(M + N + K)
    dc = (torch.rand(M, N, generator=g) + 0.1).to(dtype)
    a, w = (torch.randn(*s, generator=g).to(dtype) / 16 for s in ((M, K), (N, K)))
    inf, kept = float("inf"), [k for k in range(K) if k not in (0, 5, K - 1)]
    a2, w2, dc2 = a.clone(), w.clone(), dc.clone()
    w2[N - 1, 0], w2[0, 5], w2[N // 64 * 64 - 1, K - 1] = inf, -inf, inf
    a2[M - 1, 0], a2[0, 5], a2[M // 64 * 64 - 1, K - 1] = inf, -inf, inf
    dc2[M - 1, N - 1] = float("nan")
    rows, cols = list(range(M - 1)), list(range(N - 1))
    for pad in (0, 8, 3):
        for ws in (workspace, None):
            clean = run_backward(dc, None, a, w, "none", "f32", (pad, pad), ws)
            _, dA, dW, _ = run_backward(dc, None, a2, w2, "none", "f32", (pad, pad), ws)
            for got, ref in ((dA, clean[1]), (dW, clean[2])):
                assert torch.equal(got[:, kept], ref[:, kept]), (pad, ws is None)
                for k, x in ((0, inf), (5, -inf), (K - 1, inf)):
                    assert bool((got[:, k] == x).all()), (pad, ws is None, k)
            _, dA, dW, db = run_backward(dc2, None, a, w, "none", "f32", (pad, pad), ws)
            assert torch.equal(dA[rows], clean[1][rows]) and torch.equal(dW[cols], clean[2][cols]) and torch.equal(db[cols], clean[3][cols])
            assert bool(torch.isnan(dA[M - 1].float()).all() and torch.isnan(dW[N - 1]).all() and torch.isnan(db[N - 1])), (pad, ws is None)
