"""Forward-mode derivatives, which no operator has, are refused rather than lost: checked ahead of the device, so without a GPU."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from tiled_stage_software_amd import ops

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
X, W = torch.ones(3, 64, dtype=BF), torch.ones(40, 64, dtype=BF)
Y, S = torch.ones(3, 40, dtype=BF), torch.ones(40, dtype=torch.float32)
Q, K = torch.ones(3, 2, 8), torch.ones(3, 1, 8)
POS = torch.zeros(3, dtype=torch.int64)
COS, SIN = ops.rope_table(4, 8)
V = torch.ones(64)
CODES, SCALES = torch.zeros(40, 32, dtype=torch.uint8), torch.ones(40, 2, dtype=BF)

# an operator, and its inputs of which each in turn has a tangent
CALLS = {
    "rmsnorm": (lambda x, w, r: ops.rmsnorm(x, w, r), (X, V, X)),
    "rmsnorm to 8 bits": (lambda x, w: ops.rmsnorm(x, w, out_dtype=F8), (X, V)),
    "rmsnorm_backward": (lambda dy, h, w, r: ops.rmsnorm_backward(dy, h, w, r), (X, X, V, torch.ones(3))),
    "matmul_f8": (lambda s: ops.matmul_f8(X.to(F8), W.to(F8), None, s), (S,)),
    "matmul_w4": (lambda a, s: ops.matmul_w4(a, CODES, s, group=32), (X, SCALES)),
    "linear": (lambda x, w, b, r: ops.linear(x, w, b, "gelu", r), (X, W, S, Y)),
    "linear_keeping": (lambda x, w, b, r: ops.linear_keeping(x, w, b, "gelu", r), (X, W, S, Y)),
    "linear_backward": (lambda dy, x, w, z: ops.linear_backward(dy, x, w, z, "gelu"), (Y, X, W, Y)),
    "qk_norm_rope": (lambda q, k, a, b, c, s: ops.qk_norm_rope(q, k, a, b, POS, c, s), (Q, K, V[:8], V[:8], COS, SIN)),
    "qk_norm_rope_backward": (lambda dq, dk, q, k, a: ops.qk_norm_rope_backward(dq, dk, q, k, a, a, POS, COS, SIN), (Q, K, Q, K, V[:8])),
}


@pytest.mark.parametrize("name", CALLS)
def test_inputs_with_tangents_are_refused(name):
    call, inputs = CALLS[name]
    for i, t in enumerate(inputs):
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(t.clone(), torch.ones_like(t))
            args = list(inputs)
            args[i] = dual
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call(*args)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):   # (tangents pass there too)
                call(*args)
            leaf = forward_ad.make_dual(t.clone().requires_grad_(), torch.ones_like(t))
            args[i] = leaf
            with pytest.raises((NotImplementedError, ValueError)):   # (cos and sin take no gradient)
                call(*args)
            with pytest.raises(ValueError, match="GPU"):             # a level alone is no reason
                call(*inputs)
    with pytest.raises(ValueError, match="GPU"):
        call(*inputs)


def test_transforms_are_refused():
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda x: ops.linear(x, W), (X,), (X,))
