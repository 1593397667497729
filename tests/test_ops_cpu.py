"""The operators around the products, on the CPU: refusals before anything is launched, quick
returns, workspace sizes, and the quantisers."""
import os
import subprocess
import sys

import pytest
import torch

from tiled_stage_software_amd import libgemm as lg, ops
from ops_util import unpack4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # a fake device address: nothing here launches
F32, BF16, F16, F8 = lg.GEMM_F32, lg.GEMM_BF16, lg.GEMM_F16, lg.GEMM_F8E4M3
BAD = lg.GEMM_ERR_INVALID_ARG


def norm(**kw):
    a = dict(in_type=BF16, w_type=BF16, y_type=F8, rows=3, cols=40, eps=1e-6, x=P, ldx=40, r=P, ldr=40, w=P, h=P, ldh=40,
             y=P, ldy=40, scale=P, rstd=P)
    a.update(kw)
    return lg.gemm_rmsnorm(**a)


@pytest.mark.parametrize("kw", [
    dict(in_type=F8), dict(in_type=9), dict(w_type=F16), dict(w_type=F8), dict(y_type=7), dict(y_type=-1),
    dict(rows=-1), dict(cols=-1), dict(cols=(1 << 30) + 1), dict(rows=1 << 40), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(ldx=39), dict(ldr=39), dict(ldh=0), dict(ldy=39), dict(x=0), dict(y=0), dict(scale=0),
])
def test_norm_refuses(kw):
    assert norm(**kw) == BAD
    assert lg.gemm_last_error() != ""


@pytest.mark.parametrize("kw", [dict(rows=0, x=0, y=0, scale=0), dict(cols=0, x=0, y=0), dict(rows=0, cols=0)])
def test_norm_of_nothing(kw):
    assert norm(**kw) == lg.GEMM_OK


def bwd(**kw):
    a = dict(in_type=BF16, w_type=F32, rows=3, cols=40, dy=P, lddy=40, h=P, ldh=40, w=P, rstd=P, dh=P, lddh=40, dx=P,
             lddx=40, dw=P, workspace=P, workspace_bytes=1 << 20)
    a.update(kw)
    return lg.gemm_rmsnorm_bwd(**a)


@pytest.mark.parametrize("kw", [
    dict(in_type=F8), dict(w_type=F16), dict(rows=-2), dict(cols=-2), dict(lddy=39), dict(ldh=39), dict(lddh=39),
    dict(lddx=39), dict(dy=0), dict(h=0), dict(rstd=0), dict(dx=0), dict(workspace=P + 16),
])
def test_norm_backward_refuses(kw):
    assert bwd(**kw) == BAD
    assert lg.gemm_last_error() != ""


def test_norm_backward_of_nothing():
    assert bwd(cols=0) == lg.GEMM_OK
    assert bwd(rows=0, dw=0, dy=0, h=0, rstd=0, dx=0) == lg.GEMM_OK


def test_norm_backward_workspace():
    assert lg.gemm_rmsnorm_bwd_workspace_size(BF16, 1, 4096) == (lg.GEMM_OK, 0)       # one row: nothing to join
    s, n = lg.gemm_rmsnorm_bwd_workspace_size(BF16, 16384, 4096)
    assert s == lg.GEMM_OK and n % (4096 * 4) == 0 and 0 < n <= 64 << 20
    assert lg.gemm_rmsnorm_bwd_workspace_size(BF16, 5, 0) == (lg.GEMM_OK, 0)
    assert lg.gemm_rmsnorm_bwd_workspace_size(F8, 5, 8)[0] == BAD
    assert lg.gemm_rmsnorm_bwd_workspace_size(BF16, -1, 8)[0] == BAD


def f8(**kw):
    a = dict(M=4, N=5, K=24, alpha=1.0, A=P, lda=24, scale_a=P, B=P, ldb=24, scale_b=P, beta=0.0, C=P, c_type=BF16, ldc=5,
             workspace=P, workspace_bytes=0)
    a.update(kw)
    return lg.gemm_f8(**a)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(K=1 << 31), dict(lda=23), dict(ldb=23), dict(ldc=4), dict(A=0), dict(B=0),
    dict(C=0), dict(c_type=F8), dict(c_type=5), dict(workspace=P + 8),
])
def test_f8_refuses(kw):
    assert f8(**kw) == BAD
    assert lg.gemm_last_error() != ""


def w4(**kw):
    a = dict(in_type=BF16, M=4, N=5, K=96, group=32, alpha=1.0, A=P, lda=96, codes=P, ldw=48, scales=P, zeros=P, lds=3,
             beta=0.0, C=P, c_type=BF16, ldc=5, workspace=P, workspace_bytes=0)
    a.update(kw)
    return lg.gemm_w4(**a)


@pytest.mark.parametrize("kw", [
    dict(in_type=F32), dict(in_type=F8), dict(c_type=F16), dict(M=-1), dict(N=-1), dict(K=-1), dict(group=0),
    dict(group=16), dict(group=48), dict(group=-32), dict(lda=95), dict(ldw=47), dict(lds=2), dict(ldc=4), dict(A=0),
    dict(codes=0), dict(scales=0), dict(C=0), dict(workspace=P + 8), dict(K=97, lda=97, lds=4),
])
def test_w4_refuses(kw):
    assert w4(**kw) == BAD
    assert lg.gemm_last_error() != ""


def test_products_of_nothing():
    assert f8(M=0, A=0, C=0) == lg.GEMM_OK
    assert f8(N=0, B=0, C=0, ldc=1) == lg.GEMM_OK
    assert w4(M=0, A=0, C=0) == lg.GEMM_OK
    assert w4(N=0, codes=0, scales=0, C=0, ldc=1) == lg.GEMM_OK


def test_product_workspaces():
    for s, n in (lg.gemm_f8_workspace_size(1, 4096, 4096), lg.gemm_w4_workspace_size(BF16, 1, 4096, 4096, 128)):
        assert s == lg.GEMM_OK and 0 <= n <= 64 << 20
    assert lg.gemm_f8_workspace_size(-1, 1, 1)[0] == BAD
    assert lg.gemm_w4_workspace_size(F32, 1, 1, 1, 32)[0] == BAD
    assert lg.gemm_w4_workspace_size(BF16, 1, 1, 1, 33)[0] == BAD


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the calls pass fake device addresses that a launch would dereference")
def test_debugging_names_the_kernel():
    """GEMM_DEBUG=1: each call's sizes and kernel on stderr, before the launch (which the runtime refuses: no GPU)."""
    code = ("from tiled_stage_software_amd import libgemm as lg\n"
            "P = 0x10000\n"
            "lg.gemm_f8(1, 64, 256, 1.0, P, 256, P, P, 256, P, 0.0, P, 1, 64)\n"
            "lg.gemm_f8(300, 640, 256, 1.0, P, 256, P, P, 256, P, 0.0, P, 1, 640)\n"
            "lg.gemm_w4(1, 1, 64, 256, 128, 1.0, P, 256, P, 128, P, 0, 2, 0.0, P, 1, 64)\n"
            "lg.gemm_rmsnorm(1, 1, 3, 2, 64, 1e-6, P, 64, 0, 0, P, 0, 0, P, 64, P, P)\n")
    env = dict(os.environ, GEMM_DEBUG="1")
    err = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, cwd=ROOT).stderr
    for text in ("f8 -> type 1 M=1 N=64 K=256: few rows", "M=300 N=640 K=256: tiles", " x 128 tiles, 1 splits of K",
                 "w4 type 1 -> 1 M=1 N=64 K=256 group=128: dot products", "rmsnorm type 1 -> 3 rows=2 cols=64"):
        assert text in err, (text, err)
    env.pop("GEMM_DEBUG")
    assert "libgemm:" not in subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, cwd=ROOT).stderr


def test_wrappers_refuse_other_shapes_and_types():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.rmsnorm(x, torch.ones(7, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ops.rmsnorm(x, torch.ones(8, dtype=torch.float16))
    with pytest.raises(ValueError):
        ops.rmsnorm(x, residual=torch.zeros(2, 7, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ops.rmsnorm(x.t())
    with pytest.raises(ValueError):
        ops.rmsnorm(x, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        ops.rmsnorm_backward(x, x, None, torch.zeros(3))
    q = torch.zeros(2, 8, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        ops.matmul_f8(q, x)
    with pytest.raises(ValueError):
        ops.matmul_f8(q, q[:, :7])
    with pytest.raises(ValueError):
        ops.matmul_f8(q, q, scale_a=torch.ones(3))
    with pytest.raises(ValueError):
        ops.matmul_f8(q, q, beta=1.0)
    with pytest.raises(ValueError):
        ops.matmul_w4(x, torch.zeros(3, 5, dtype=torch.uint8), torch.ones(3, 1, dtype=torch.bfloat16), group=32)
    with pytest.raises(ValueError):
        ops.matmul_f8(q, q, C=torch.zeros(1, 2).expand(2, 2))  # rows that lie on each other


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("k", [64, 97])
def test_quantize_w4_is_half_a_step_off(k, zeros):
    g = torch.Generator().manual_seed(k)
    w = torch.randn(6, k, generator=g) + (0.5 if zeros else 0.0)
    codes, s, z = ops.quantize_w4(w, 32, torch.float32, zeros)
    assert codes.shape == (6, (k + 1) // 2) and s.shape == (6, -(-k // 32)) and (z is not None) == zeros
    each = lambda t: t.repeat_interleave(32, 1)[:, :k]  # noqa: E731
    back = each(s) * (unpack4(codes, k).float() - (each(z) if zeros else 8.0))
    # codes are rounded (half a step) and clamped: the largest value may lie half a step past 15
    # (centred: 8 + 7.5; with zeros the rounding of the zero point)
    assert bool(((back - w).abs() <= 1.01 * each(s)).all())
    assert float(((back - w).abs() <= 0.51 * each(s)).float().mean()) > 0.9


def test_quantize_f8():
    t = torch.tensor([[0.0, 0.0], [448.0, -1.0], [1e-3, 2e-3]])
    q, s = ops.quantize_f8(t)
    assert s[0] == ops.TINY and s[1] == 1.0
    assert torch.equal(q[:2].float(), t[:2])
    assert bool(((q.float() * s[:, None] - t).abs() <= 2.0 ** -4 * t.abs()).all())


no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the calls pass fake device addresses that a launch would dereference")


def notes(calls):
    """What GEMM_DEBUG prints for these calls of lg.* at fake addresses (P), before the launch that the runtime refuses."""
    code = f"from tiled_stage_software_amd import libgemm as lg\nP = {P}\n" + "\n".join(calls)
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, GEMM_DEBUG="1"), capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    return r.stderr


@no_gpu
@pytest.mark.parametrize("M,N,K,loads", [
    (256, 512, 8388481, "direct loads of copied rows"),   # 128 rows of 2 * 8388544 bytes: just below 2^31
    (256, 512, 8388609, "staged loads"), (256, 512, 17000001, "staged loads"), (256, 512, 17000064, "staged loads"),
    (64, 128, 16777089, "direct loads of copied rows"), (64, 128, 35000001, "staged loads"),
    (256, 512, 8388544, "direct loads\n"), (256, 512, 8388608, "staged loads"),
])
def test_w4_rows_whose_copies_pass_32_bits_are_not_copied(M, N, K, loads):
    """The direct loads hold a row's offset in its tile in 32 bits, also in a copy; longer rows take the staged loads,
    and no workspace is asked for a copy of them."""
    groups = -(-K // 128)
    s, nbytes = lg.gemm_w4_workspace_size(BF16, M, N, K, 128)
    err = notes([f"lg.gemm_w4(1, {M}, {N}, {K}, 128, 1.0, P, {K}, P, {(K + 1) // 2}, P, P, {groups}, 0.0, P, 1, {N}, P, {nbytes})"])
    assert s == lg.GEMM_OK and f"K={K} group=128: tiles" in err and loads in err, err
    copies = M * -(-K // 64) * 128 + N * -(-K // 64) * 32
    assert (nbytes >= copies) == ("copied" in loads)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k", [64, 75])
def test_quantize_w4_of_groups_far_from_zero(t, k):
    """Zero points are whole numbers from 0 to 15, whatever the group: one value, values far from zero, zeros.  A value is
    off by half a step for its code and, at the end of the codes, half a step for the rounding of the zero point, plus
    what the scale's own rounding moves fifteen steps by."""
    g = torch.Generator().manual_seed(k)
    noise = 2 * torch.rand(12, k, generator=g) - 1
    mid = torch.tensor([5.0, -5.0, 4096.0, 6.0, 1.0, 1.0, -1.0, 0.0, 0.0, 3.0, 0.25, -0.5])
    wide = torch.tensor([0.0, 0.0, 0.0, 1e-4, 1e-3, 1e-2, 0.1, 0.0, 1.0, 3.0, 0.3, 2.0])
    w = mid[:, None] + wide[:, None] * noise
    codes, s, z = ops.quantize_w4(w, 32, t, True)
    assert bool((z == z.round()).all()) and bool(((z >= 0) & (z <= 15)).all())
    each = lambda v: v.float().repeat_interleave(32, 1)[:, :k]  # noqa: E731
    back = each(s) * (unpack4(codes, k).float() - each(z))
    steps = 0.5 + 15 * torch.finfo(t).eps / 2 + 1e-3
    assert float(((back - w).abs() / each(s)).max()) <= steps
    reach = torch.maximum(w.amax(1), torch.zeros(12)) - torch.minimum(w.amin(1), torch.zeros(12))
    assert bool((s.float() <= (reach / 15).clamp_min(torch.finfo(t).tiny)[:, None] * (1 + torch.finfo(t).eps)).all())


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    """A stream's handle does not name a device (0 is each one's default stream): the call makes its tensors' device the
    current one, and the caller's again."""
    at = [0]

    class Device:
        def __init__(self, d):
            self.index = d.index

        def __enter__(self):
            self.before, at[0] = at[0], self.index

        def __exit__(self, *error):
            at[0] = self.before

    class Stream:
        cuda_stream = 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "device", Device)
    for stream in (None, 0):
        for index in (0, 1):
            with lg.Running(stream, torch.device("cuda", index)) as on:
                assert at[0] == index and on.handle == 0
            assert at[0] == 0
    with pytest.raises(KeyError):
        with lg.Running(None, torch.device("cuda", 1)):
            raise KeyError
    assert at[0] == 0


def test_workspaces_have_to_be_whole_memory():
    """A call uses all bytes from a workspace's first to as many as it has elements: in a strided view those are others'."""
    big = torch.zeros(64, 64, dtype=torch.uint8)
    assert ops._workspace(big[3:5], None, big.device)[1:] == (big.data_ptr() + 192, 128)
    for view in (big[:, :8], big[::2], big.t()[:5], big[:1].expand(4, 64)):
        with pytest.raises(ValueError, match="contiguous"):
            ops._workspace(view, None, big.device)
    with pytest.raises(ValueError, match="contiguous"):
        lg.workspace_of(big[:, :8], big.device)


@no_gpu
@pytest.mark.parametrize("call", [
    "lg.gemm_w4(1, 1 << 30, 64, 32, 32, 1.0, P, 32, P, 16, P, 0, 1, 0.0, P, 1, 64)",
    "lg.gemm_w4(1, 5, 1 << 30, 32, 32, 1.0, P, 32, P, 16, P, 0, 1, 0.0, P, 1, 1 << 30)",
    "lg.gemm_w4(1, 1, 1 << 30, 32, 32, 1.0, P, 32, P, 16, P, 0, 1, 0.0, P, 1, 1 << 30)",
    "lg.gemm_f8(1 << 30, 1 << 30, 16, 1.0, P, 16, 0, P, 16, 0, 0.0, P, 1, 1 << 30)",
    "lg.gemm_f8(5, 1 << 30, 16, 1.0, P, 16, 0, P, 16, 0, 0.0, P, 1, 1 << 30)",
    "lg.gemm_f8(1 << 30, 1 << 30, 1 << 20, 1.0, P, 1 << 20, 0, P, 1 << 20, 0, 0.0, P, 1, 1 << 30)",
])
def test_every_size_is_launched(call):
    """The largest sizes pass the limits of one grid: they go out in several launches, and nothing but the missing device is
    in their way."""
    err = notes([call])
    assert "no ROCm-capable device" in err and "invalid" not in err, err


@no_gpu
def test_workspaces_asked_for_are_used_and_enough():
    """With the bytes of the query a call does what it would with any more; and where the query asks for some, a call of
    one of the result types does something with them."""
    g = torch.Generator().manual_seed(1)
    draw = lambda low, high: int(round(low * (high / low) ** float(torch.rand(1, generator=g))))  # noqa: E731
    shapes = [(256, 512, 17000001), (64, 100, 100), (40, 4096, 64), (333, 3001, 2049), (64, 128, 8388608), (1 << 30, 1 << 30, 1 << 30),
              (33, 14336, 4096), (300, 520, 1000), (129, 260, 16000), (200, 300, 15000), (17, 14336, 4097), (300, 300, 40)]
    shapes += [(draw(1, 4096), draw(16, 16384), draw(16, 16384)) for _ in range(60)]
    calls, sizes = [], []
    big = (1 << 62) - 1
    for M, N, K in shapes:
        s, f = lg.gemm_f8_workspace_size(M, N, K)
        s4, w = lg.gemm_w4_workspace_size(BF16, M, N, K, 64)
        assert s == s4 == lg.GEMM_OK
        sizes.append((f, w))
        for ws in (0, f, big):
            for t in (1, 0):
                calls.append(f"lg.gemm_f8({M}, {N}, {K}, 1.0, P, {K}, 0, P, {K}, 0, 0.0, P, {t}, {N}, P, {ws})")
        for ws in (0, w, big):
            calls.append(f"lg.gemm_w4(1, {M}, {N}, {K}, 64, 1.0, P, {K}, P, {(K + 1) // 2}, P, P, {-(-K // 64)}, 0.0, P, 1, {N}, P, {ws})")
    said = []
    for line in notes(calls).splitlines():
        if " M=" in line:
            said.append(line.split(": ", 2)[2])
        elif "status" not in line:
            said[-1] += line
    assert len(said) == 9 * len(shapes)
    for i, (f, w) in enumerate(sizes):
        none, asked, more = said[9 * i:9 * i + 2], said[9 * i + 2:9 * i + 4], said[9 * i + 4:9 * i + 6]
        assert asked == more, (shapes[i], asked, more)
        assert (f > 0) == (asked != none), (shapes[i], f, none, asked)
        none, asked, more = said[9 * i + 6:9 * i + 9]
        assert asked == more, (shapes[i], asked, more)
        assert (w > 0) == (asked != none), (shapes[i], w, none, asked)


def test_the_package_has_the_operators():
    import tiled_stage_software_amd as pkg
    assert pkg.ops is ops and pkg.GEMM_F8E4M3 == lg.GEMM_F8E4M3
    code = "import sys, tiled_stage_software_amd as p; p.ops, p.GEMM_F8E4M3; assert 'torch' not in sys.modules"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
