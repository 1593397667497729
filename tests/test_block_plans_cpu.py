"""What the backward pass of the product with bias, activation and residual launches, without a GPU: its plan is said whole before the
first launch, the workspace that it asks for is enough, the largest sizes reach their products' launches, and the sizes that the large
tiles are tested on take them."""
import pytest
import torch

import test_gpu_block_large as large
from test_block_cpu import BF16, OK, backward_call, linear_call, no_gpu, notes
from tiled_stage_software_amd import libgemm as lg

MANY = 1 << 40


def plain_call(M, N, K, ws=0, need=(1, 1), dw=1):
    """A call without an activation, on dC in place of dZ and without db: its first launch is the products'."""
    return (f"lg.gemm_linear_bwd(1, {M}, {N}, {K}, 0, P, 1, {N}, 0, {N}, P, {K}, P, {K}, 0, {N}, P * {need[0]}, {K}, P * {need[1]}, {dw}, {K}, 0, "
            f"P, {ws})")


@no_gpu
@pytest.mark.parametrize("call,said", [
    (backward_call(4096, 14336, 4096, MANY), ["dZ in 36 parts\n", "4096 x 4096 x 14336: 256 x 256 tiles", "14336 x 4096 x 4096: 256 x 256 tiles"]),
    (backward_call(513, 1001, 643, MANY), ["parts, dZ copied, A copied, W copied\n", "513 x 643 x 1001: 64 x 128 tiles", "1001 x 643 x 513: 128 x 128"]),
    (backward_call(513, 1001, 643, 0), ["dZ in 1 parts\n", "513 x 643 x 1001: as a 16-bit product", "1001 x 643 x 513: as a 16-bit product"]),
    (plain_call(64, 64, 8192, 0, (0, 1)), ["64 x 8192 x 64: 128 x 128 tiles, 1 splits"]),
])
def test_plans_are_said_before_the_first_launch(call, said):
    err = notes([call])
    for text in said:
        assert text in err, (text, err)


@no_gpu
def test_backward_workspace_is_enough():
    """With the bytes of the query a call of contiguous operands does what it would with any more, whichever gradients it is asked
    for; every line compared says a plan."""
    g = torch.Generator().manual_seed(2)
    draw = lambda low, high: int(round(low * (high / low) ** float(torch.rand(1, generator=g))))  # noqa: E731
    shapes = [(4096, 14336, 4096), (513, 1001, 643), (100, 33, 65), (1, 1, 1), (7, 9, 33), (8192, 64, 64), (64, 8192, 8192)]
    shapes += [(draw(1, 8192), draw(8, 16384), draw(8, 16384)) for _ in range(60)]
    shapes += [(draw(1, 8192) // 8 * 8 + 8, draw(8, 16384) // 8 * 8, draw(8, 16384) // 8 * 8) for _ in range(30)]
    calls, used = [], 0
    for M, N, K in shapes:
        s, b = lg.gemm_linear_bwd_workspace_size(BF16, M, N, K)
        assert s == OK
        for call in (backward_call, plain_call):
            calls += [f"import sys; sys.stderr.write('libgemm: call\\n')\n{call(M, N, K, ws)}" for ws in (b, (1 << 62) - 1, 0)]
    said = [[line for line in part.splitlines() if "status" not in line] for part in notes(calls).split("libgemm: call\n")[1:]]
    assert len(said) == 6 * len(shapes)
    for i, shape in enumerate(shapes):
        for asked, more, none in (said[6 * i:6 * i + 3], said[6 * i + 3:6 * i + 6]):
            assert asked == more and len(asked) == 3 and "linear_bwd" in asked[0] and all("tiles" in line for line in asked[1:]), (shape, asked, more)
            used += asked != none
    assert used > len(shapes)


@no_gpu
@pytest.mark.parametrize("call,said", [
    (plain_call(1 << 26, 512, 64, MANY), "tiles"),
    (plain_call(1 << 30, 512, 64, MANY), "as a 16-bit product"),
    (plain_call(8, 16, 1 << 30, MANY), "as a 16-bit product"),          # (pitches that the tiles' offsets do not hold)
    (plain_call(1 << 30, 64, 64, 0, (1, 0)), "as a 16-bit product"),    # (more tiles than a launch counts)
    (plain_call(8, 1 << 21, 64, MANY, (1, 1)), "tiles"),
    (plain_call(4096, 1 << 21, 1 << 21, MANY, (1, 0)), "tiles"),
    (plain_call(1 << 30, 1 << 30, 8, 0, (1, 0)), "as a 16-bit product"),
    (plain_call(7, 9, 33), "as a 16-bit product"),
])
def test_the_largest_products_are_launched(call, said):
    err = notes([call])
    assert said in err and "no ROCm-capable device" in err and "invalid" not in err, err


@no_gpu
@pytest.mark.parametrize("shapes,tile", [(large.LINEAR_256, "256 x 256"), (large.LINEAR_192, "192 x 256")])
def test_sizes_of_the_large_tiles(shapes, tile):
    for M, N, K in shapes:
        for pad in (0, 8):
            assert f"  {tile} tiles, 1 splits of K, direct loads\n" in notes([linear_call(M, N, K, 0, K + pad, K + pad)])
    assert any(f"  {tile} tiles, 1 splits of K, direct loads of copied rows" in notes([linear_call(*s, large.WS, s[2] + 3, s[2] + 1)]) for s in shapes)


@no_gpu
def test_backward_sizes_of_the_large_tiles():
    for shapes, of_a, of_w in ((large.GRAD_A, True, False), (large.GRAD_W, False, True), (large.GRAD_BOTH, True, True)):
        for M, N, K in shapes:
            err = notes([backward_call(M, N, K, large.WS)])
            assert (f"  {M} x {K} x {N}: 256 x 256 tiles" in err) == of_a and (f"  {N} x {K} x {M}: 256 x 256 tiles" in err) == of_w, err
