"""The product with bias, activation and residual, and the norm and rotation of heads, on the CPU: refusals before anything is
launched, calls of nothing, workspace sizes, what is launched, and the wrappers' checks."""
import math
import os
import subprocess
import sys

import pytest
import torch

from tiled_stage_software_amd import libgemm as lg, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # a fake device address: nothing here launches
F32, BF16, F16, F8 = lg.GEMM_F32, lg.GEMM_BF16, lg.GEMM_F16, lg.GEMM_F8E4M3
OK, BAD = lg.GEMM_OK, lg.GEMM_ERR_INVALID_ARG
GELU, RELU, NONE = lg.GEMM_ACT_GELU, lg.GEMM_ACT_RELU, lg.GEMM_ACT_NONE
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the calls pass fake device addresses that a launch would dereference")


def refused(status):
    assert status == BAD
    assert lg.gemm_last_error() != ""


def linear(**kw):
    a = dict(in_type=BF16, M=3, N=40, K=24, A=P, lda=24, W=P, ldw=24, bias=P, bias_type=BF16, act=GELU, R=P, ldr=40, Z=P, ldz=40,
             C=P, c_type=BF16, ldc=40, workspace=P, workspace_bytes=0)
    a.update(kw)
    return lg.gemm_linear(**a)


@pytest.mark.parametrize("kw", [
    dict(in_type=F32), dict(in_type=F8), dict(in_type=9), dict(c_type=F16), dict(c_type=F8), dict(bias_type=F16), dict(bias_type=7),
    dict(act=-1), dict(act=5), dict(M=-1), dict(N=-1), dict(K=-1), dict(M=(1 << 30) + 1), dict(N=1 << 40), dict(K=1 << 31),
    dict(lda=23), dict(ldw=23), dict(ldc=39), dict(ldr=39), dict(ldz=39), dict(ldz=0), dict(A=0), dict(W=0), dict(C=0), dict(workspace=P + 16),
])
def test_linear_refuses(kw):
    refused(linear(**kw))


@pytest.mark.parametrize("kw", [dict(M=0, A=0, C=0), dict(N=0, W=0, C=0), dict(M=0, N=0, K=0, A=0, W=0, C=0)])
def test_linear_of_nothing(kw):
    assert linear(**kw) == OK


def linear_bwd(**kw):
    a = dict(in_type=BF16, M=3, N=40, K=24, act=GELU, dC=P, dc_type=BF16, lddc=40, Z=P, ldz=40, A=P, lda=24, W=P, ldw=24, dZ=P, lddz=40,
             dA=P, ldda=24, dW=P, dw_type=BF16, lddw=24, dbias=P, workspace=P, workspace_bytes=0)
    a.update(kw)
    return lg.gemm_linear_bwd(**a)


@pytest.mark.parametrize("kw", [
    dict(in_type=F32), dict(in_type=F8), dict(dc_type=F16), dict(dw_type=F16), dict(dw_type=-1), dict(act=5), dict(M=-1), dict(N=-1), dict(K=-1),
    dict(lddc=39), dict(ldz=39), dict(lddz=39), dict(lda=23), dict(ldw=23), dict(ldda=23), dict(lddw=23), dict(dC=0), dict(Z=0), dict(A=0),
    dict(W=0), dict(dZ=0), dict(dZ=0, dA=0), dict(dZ=0, dW=0), dict(dZ=0, act=NONE, dc_type=F32), dict(workspace=P + 128),
])
def test_linear_backward_refuses(kw):
    refused(linear_bwd(**kw))


@pytest.mark.parametrize("kw", [
    dict(N=0, dA=0, dC=0, Z=0, dZ=0), dict(M=0, N=0, A=0, W=0), dict(M=0, N=0, K=0),
])
def test_linear_backward_of_nothing(kw):
    assert linear_bwd(**kw) == OK


def test_linear_workspaces():
    for size in (lg.gemm_linear_workspace_size, lg.gemm_linear_bwd_workspace_size):
        for bad in ((F32, 1, 1, 1), (F8, 1, 1, 1), (BF16, -1, 1, 1), (BF16, 1, -1, 1), (BF16, 1, 1, -1)):
            assert size(*bad)[0] == BAD
        for none in ((BF16, 0, 64, 64), (BF16, 64, 0, 64)):
            assert size(*none) == (OK, 0)
    assert lg.gemm_linear_workspace_size(BF16, 64, 64, 0) == (OK, 0)
    assert lg.gemm_linear_workspace_size(F16, 1, 14336, 4096) == (OK, 0)        # few rows
    s, n = lg.gemm_linear_workspace_size(F16, 64, 128, 16384)                   # splits of a long K
    assert s == OK and 64 * 128 * 4 * 2 <= n <= 64 << 20
    s, n = lg.gemm_linear_bwd_workspace_size(BF16, 4096, 14336, 4096)
    assert s == OK and 0 < n <= 64 << 20 and n % 256 == 0
    s, n = lg.gemm_linear_bwd_workspace_size(BF16, 100, 33, 65)                 # all three copied
    assert s == OK and n >= 2 * (100 * 33 + 100 * 65 + 33 * 65)


def heads(ld=120, hs=40, at=P):
    return lg.GemmHeads(at, ld, hs)


def rope(**kw):
    a = dict(positions=P, cos=P, sin=P, ld=8, rows=100, rot_dim=16, pairs=lg.GEMM_ROPE_HALVES)
    a.update(kw)
    return lg.GemmRope(*a.values())


def qk(**kw):
    a = dict(in_type=BF16, w_type=BF16, tokens=5, q_heads=3, k_heads=2, head_dim=40, eps=1e-6, q=heads(), k=heads(), wq=P, wk=P, rope=rope(),
             out_q=heads(), out_k=heads())
    a.update(kw)
    return lg.gemm_qk_norm_rope(**a)


def qk_bwd(**kw):
    a = dict(in_type=BF16, w_type=BF16, tokens=5, q_heads=3, k_heads=2, head_dim=40, eps=1e-6, dq=heads(), dk=heads(), q=heads(), k=heads(),
             wq=P, wk=P, rope=rope(), dxq=heads(), dxk=heads(), dwq=P, dwk=P, workspace=P, workspace_bytes=1 << 16)
    a.update(kw)
    return lg.gemm_qk_norm_rope_bwd(**a)


SAME = [
    dict(in_type=F8), dict(in_type=8), dict(w_type=F16), dict(w_type=F8), dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(q_heads=-1),
    dict(k_heads=-1), dict(q_heads=65537), dict(head_dim=0), dict(head_dim=-4), dict(head_dim=1025), dict(eps=-1.0), dict(eps=math.inf),
    dict(eps=math.nan), dict(q=None), dict(k=None), dict(q=heads(at=0)), dict(k=heads(at=0)),
    dict(q=heads(119)), dict(q=heads(hs=39)), dict(q=heads(0)), dict(q=heads(hs=0)), dict(q=heads(-120)), dict(q=heads(hs=-40)),
    dict(k=heads(79)), dict(q=heads(1 << 41)), dict(q=heads(39, 200)), dict(q=heads(40, 199)),
    dict(rope=rope(rot_dim=15)), dict(rope=rope(rot_dim=42, ld=21)), dict(rope=rope(rot_dim=-2)), dict(rope=rope(ld=7)), dict(rope=rope(rows=-1)),
    dict(rope=rope(pairs=2)), dict(rope=rope(pairs=-1)), dict(rope=rope(positions=0)), dict(rope=rope(cos=0)), dict(rope=rope(sin=0)),
]


@pytest.mark.parametrize("kw", SAME + [dict(out_q=None), dict(out_k=heads(at=0)), dict(out_q=heads(100)), dict(out_k=heads(hs=7))])
def test_heads_refuse(kw):
    refused(qk(**kw))


@pytest.mark.parametrize("kw", SAME + [dict(dq=None), dict(dk=heads(at=0)), dict(dq=heads(100)), dict(dxq=None), dict(dxk=heads(hs=39)),
                                       dict(workspace=P + 64)])
def test_heads_backward_refuses(kw):
    refused(qk_bwd(**kw))


@pytest.mark.parametrize("kw", [dict(tokens=0, q=None, k=None), dict(q_heads=0, k_heads=0, q=None, k=None), dict(tokens=0, rope=None)])
def test_heads_of_nothing(kw):
    assert qk(out_q=None, out_k=None, **kw) == OK
    assert qk_bwd(dq=None, dk=None, dxq=None, dxk=None, dwq=0, dwk=0, **kw) == OK


def test_heads_workspace():
    size = lg.gemm_qk_norm_rope_bwd_workspace_size
    assert size(BF16, 1, 1, 0, 128) == (OK, 0)   # one head: nothing to join
    assert size(BF16, 0, 4, 4, 128) == (OK, 0)
    s, n = size(BF16, 8192, 32, 8, 128)
    assert s == OK and n % (128 * 4) == 0 and 0 < n <= 4 << 20
    for bad in ((F8, 1, 1, 1, 8), (BF16, -1, 1, 1, 8), (BF16, 1, -1, 1, 8), (BF16, 1, 1, -1, 8), (BF16, 1, 1, 1, 0), (BF16, 1, 1, 1, 1025)):
        assert size(*bad)[0] == BAD


# ------------------------------------------------------------------ what is launched
def notes(calls):
    """What GEMM_DEBUG prints for these calls of lg.* at fake addresses (P), before the launch that the runtime refuses."""
    head = (f"from tiled_stage_software_amd import libgemm as lg\nP = {P}\nH = lg.GemmHeads\nR = lg.GemmRope\n")
    r = subprocess.run([sys.executable, "-c", head + "\n".join(calls)], env=dict(os.environ, GEMM_DEBUG="1"), capture_output=True,
                       text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    return r.stderr


def linear_call(M, N, K, ws=0, lda=None, ldw=None, c=1):
    return f"lg.gemm_linear(1, {M}, {N}, {K}, P, {lda or K}, P, {ldw or K}, 0, 0, 2, 0, 0, 0, 0, P, {c}, {N}, P, {ws})"


def backward_call(M, N, K, ws=0, act=2, c=1):
    return (f"lg.gemm_linear_bwd(1, {M}, {N}, {K}, {act}, P, {c}, {N}, P, {N}, P, {K}, P, {K}, P, {N}, P, {K}, P, 1, {K}, P, P, {ws})")


@no_gpu
@pytest.mark.parametrize("call,said", [
    (linear_call(1, 4096, 4096), "M=1 N=4096 K=4096 act=2: few rows"),
    (linear_call(32, 32768, 2048, 1 << 40), ": tiles"),
    (linear_call(32, 352, 16000, 1 << 40), ": tiles"),
    (linear_call(32, 352, 16000), ": few rows"),                                # (tiles ask for a workspace there)
    (linear_call(33, 4096, 63), ": 128 x 128 tiles"),
    (linear_call(40, 4096, 0, 0, 1, 1), ": 128 x 128 tiles"),
    (linear_call(4096, 4096, 14336), "256 x 256 tiles, 1 splits of K, direct loads\n"),
    (linear_call(333, 3001, 2049), "staged loads"),
    (linear_call(64, 128, 16384, 1 << 40), "64 x 128 tiles, "),
    (linear_call(64, 128, 16384, 64), "1 splits of K, direct loads\n"),
    (linear_call(256, 512, 1 << 22, 1 << 50), ": 128 x 128 tiles"),             # rows that 32-bit offsets in a tile do not hold
    ("lg.gemm_qk_norm_rope(1, 1, 5, 3, 2, 40, 1e-6, H(P, 120, 40), H(P, 80, 40), P, P, R(P, P, P, 8, 9, 16, 0), H(P, 120, 40), H(P, 80, 40))",
     "qk_norm_rope type 1 tokens=5 heads=3+2 dim=40 rot=16"),
])
def test_debugging_names_the_kernel(call, said):
    err = notes([call])
    assert said in err, err


@no_gpu
@pytest.mark.parametrize("call", [
    linear_call(1 << 30, 64, 32), linear_call(5, 1 << 30, 32), linear_call(1 << 30, 1 << 30, 16), linear_call(1 << 30, 1 << 30, 1 << 20),
    linear_call(300, 1 << 30, 64), linear_call(100, 100, 1 << 30), linear_call(1, 1 << 30, 1 << 30), linear_call(1 << 30, 1, 1 << 21),
    backward_call(1 << 30, 1, 1), backward_call(1, 1 << 30, 16), backward_call(1 << 30, 512, 64, 1 << 50),
    backward_call(8, 16, 1 << 30, 1 << 50), backward_call(7, 9, 33, 0), backward_call(7, 9, 33, 1 << 20),
    "lg.gemm_qk_norm_rope(1, 1, 1 << 30, 65536, 65536, 1024, 1e-6, H(P, 1 << 26, 1024), H(P, 1 << 26, 1024), P, P, None, H(P, 1 << 26, 1024), H(P, 1 << 26, 1024))",
    "lg.gemm_qk_norm_rope(0, 0, 1 << 30, 2, 1, 1, 1e-6, H(P, 2, 1), H(P, 1, 1), P, P, None, H(P, 1, 1 << 30), H(P, 1, 1))",
    "lg.gemm_qk_norm_rope_bwd(1, 1, 1 << 30, 2, 1, 64, 1e-6, H(P, 128, 64), H(P, 64, 64), H(P, 128, 64), H(P, 64, 64), P, P, None, H(P, 128, 64), H(P, 64, 64), P, P, P, 1 << 30)",
])
def test_every_size_is_launched(call):
    """The largest sizes pass the limits of one grid or of a tile's offsets: nothing but the missing device is in their way."""
    err = notes([call])
    assert "no ROCm-capable device" in err and "invalid" not in err, err


@no_gpu
def test_workspaces_asked_for_are_used_and_enough():
    """With the bytes of the query a call of contiguous operands does what it would with any more; and what it does without
    any is something else only where the query asks for some."""
    g = torch.Generator().manual_seed(1)
    draw = lambda low, high: int(round(low * (high / low) ** float(torch.rand(1, generator=g))))  # noqa: E731
    shapes = [(256, 512, 17001), (64, 100, 100), (40, 4096, 64), (333, 3001, 2049), (33, 14336, 4096), (300, 520, 1000), (129, 260, 16000),
              (32, 32768, 2048), (16, 352, 16000), (5, 1152, 12608), (17, 14336, 4097), (300, 300, 40), (4096, 4096, 4001)]
    shapes += [(draw(1, 4096), draw(16, 16384), draw(16, 16384)) for _ in range(60)]
    calls, sizes, big = [], [], (1 << 62) - 1
    for M, N, K in shapes:
        s, f = lg.gemm_linear_workspace_size(BF16, M, N, K)
        s2, b = lg.gemm_linear_bwd_workspace_size(BF16, M, N, K)
        assert s == s2 == OK
        sizes.append(f)
        calls += ["import sys; sys.stderr.write('libgemm: call\\n')"] + [linear_call(M, N, K, ws) for ws in (0, f, big)]
        calls += [backward_call(M, N, K, ws) for ws in (b, big)]
    said = []
    for line in notes(calls).splitlines():
        if "libgemm: call" in line:
            said.append([])
        elif " M=" in line and "linear" in line:
            said[-1].append(line.split("linear", 1)[1])
        elif "status" not in line and said:
            said[-1][-1] += line
    assert len(said) == len(shapes)
    for shape, f, (none, asked, more, backward, backward_more) in zip(shapes, sizes, said):
        assert asked == more, (shape, asked, more)
        assert asked == none or f > 0, (shape, f, none, asked)
        assert backward == backward_more, (shape, backward, backward_more)


# ------------------------------------------------------------------ wrappers
def test_wrappers_refuse_other_shapes_and_types():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    y = torch.zeros(2, 6, dtype=torch.bfloat16)
    for bad in (lambda: ops.linear(x, w[:, :7]), lambda: ops.linear(x, w.half()), lambda: ops.linear(x.t(), w), lambda: ops.linear(x[0], w),
                lambda: ops.linear(x, w, act="swish"), lambda: ops.linear(x, w, torch.zeros(5, dtype=torch.bfloat16)),
                lambda: ops.linear(x, w, torch.zeros(6, dtype=torch.float16)), lambda: ops.linear(x, w, residual=y.float()),
                lambda: ops.linear(x, w, residual=y[:, :5]), lambda: ops.linear(x, w, residual=y, out_dtype=torch.float32),
                lambda: ops.linear(x, w, out_dtype=torch.int8), lambda: ops.linear(x, w.t().contiguous().t()),
                lambda: ops.linear(x, w),                                                      # (on the CPU: nothing falls back)
                lambda: ops.linear_backward(y, x, w, None, "gelu"), lambda: ops.linear_backward(y[:1], x, w),
                lambda: ops.linear_backward(y, x, w, y.float(), "relu"), lambda: ops.linear_backward(y, x, w, workspace=3)):
        with pytest.raises(ValueError):
            bad()
    q, k = torch.zeros(3, 2, 8), torch.zeros(3, 1, 8)
    pos = torch.zeros(3, dtype=torch.int64)
    cos, sin = ops.rope_table(10, 4)
    for bad in (lambda: ops.qk_norm_rope(q, k[:2]), lambda: ops.qk_norm_rope(q, k[..., :4]), lambda: ops.qk_norm_rope(q, k.half()),
                lambda: ops.qk_norm_rope(q, k, torch.ones(7)), lambda: ops.qk_norm_rope(q, k, torch.ones(8), torch.ones(8).half()),
                lambda: ops.qk_norm_rope(q, k, positions=pos), lambda: ops.qk_norm_rope(q, k, None, None, pos.int(), cos, sin),
                lambda: ops.qk_norm_rope(q, k, None, None, pos[:2], cos, sin), lambda: ops.qk_norm_rope(q, k, None, None, pos, cos, sin[:5]),
                lambda: ops.qk_norm_rope(q, k, None, None, pos, cos.double(), sin), lambda: ops.qk_norm_rope(q, k, pairs="odd"),
                lambda: ops.qk_norm_rope(q, k, None, None, pos, cos.requires_grad_(), sin), lambda: ops.qk_norm_rope(q[0], k),
                lambda: ops.qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2)), lambda: ops.qk_norm_rope(q, k),
                lambda: ops.qk_norm_rope_backward(q[:2], k, q, k), lambda: ops.qk_norm_rope_backward(q, k.half(), q, k)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("rot", [2, 64, 90])
def test_rope_table(rot):
    """Within a rounding of fp32 of the angles' cosines and sines (taken in 64 bits, whose angles are good to 2^-53 * 40000)."""
    cos, sin = ops.rope_table(40000, rot, 10000.0)
    assert cos.shape == sin.shape == (40000, rot // 2) and cos.dtype == sin.dtype == torch.float32
    for p in (0, 1, 777, 39999):
        for i in {0, 1, rot // 4, rot // 2 - 1} & set(range(rot // 2)):
            angle = p * 10000.0 ** (-2 * i / rot)
            assert abs(float(cos[p, i]) - math.cos(angle)) <= 2.0 ** -24 and abs(float(sin[p, i]) - math.sin(angle)) <= 2.0 ** -24
