"""One MLP block of a language model through libgemm's operators, served and trained.

Serving, a prompt and then single tokens:
    h = x + residual,  y = rmsnorm(h) in 8 bits with a scale per row      (gemm_rmsnorm)
    wide = y Wu^T, the widening layer in 8 bits                            (gemm_f8)
    out = relu(wide) Wd^T, the narrowing layer with 4-bit weights          (gemm_w4)
Training, the norm's part of a step: dx, dw from the gradients of y and h  (gemm_rmsnorm_bwd)

The decoding step is captured into a graph and replayed.  Needs one GPU:
    python examples/mlp_block.py [--width 4096] [--wide 14336] [--prompt 2048] [--tokens 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tiled_stage_software_amd import ops  # noqa: E402


class Block:
    """Weights quantised once; workspaces kept, so that a call allocates nothing but its results."""

    def __init__(self, width, wide, group=128, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.norm = (1 + 0.1 * randn(width)).bfloat16()
        self.up, self.up_scale = ops.quantize_f8(randn(wide, width) / width ** 0.5)
        self.down = randn(width, wide) / wide ** 0.5
        self.codes, self.scales, self.zeros = ops.quantize_w4(self.down, group, torch.bfloat16, zeros=True)
        self.group = group
        self.ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def forward(self, x, residual):
        n = ops.rmsnorm(x, self.norm, residual, out_dtype=torch.float8_e4m3fn)
        wide = ops.matmul_f8(n.y, self.up, n.scale, self.up_scale, workspace=self.ws)
        return ops.matmul_w4(wide.relu_(), self.codes, self.scales, self.zeros, self.group, workspace=self.ws), n

    def plain(self, x, residual):
        """The same with fp32 products of the unquantised narrowing layer."""
        h = (x.float() + residual.float()).bfloat16().float()
        y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * self.norm.float()
        wide = y @ (self.up.float() * self.up_scale[:, None]).t()
        return wide.relu() @ self.down.t()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--wide", type=int, default=14336)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args(argv)
    block = Block(a.width, a.wide)
    x = torch.randn(a.prompt, a.width, device="cuda").bfloat16()
    r = torch.randn(a.prompt, a.width, device="cuda").bfloat16()
    out, n = block.forward(x, r)
    off = float((out.float() - block.plain(x, r)).norm() / block.plain(x, r).norm())
    print(f"prompt of {a.prompt}: {off:.3f} from the unquantised block")   # 4 bits: about a tenth

    # a decoding step, captured once
    x1, r1 = x[:1].clone(), r[:1].clone()
    block.forward(x1, r1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out1, n1 = block.forward(x1, r1)
    start = time.perf_counter()
    for _ in range(a.tokens):
        graph.replay()
        x1.copy_(out1)
        r1.copy_(n1.h)
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens: {(time.perf_counter() - start) / a.tokens * 1e6:.1f} us each")

    # the norm's part of a training step
    dy, dh = torch.randn_like(n.h), torch.randn_like(n.h)
    dx, dw = ops.rmsnorm_backward(dy, n.h, block.norm, n.rstd, dh, workspace=block.ws)
    print(f"gradients: |dx| {float(dx.float().norm()):.4g}, |dw| {float(dw.norm()):.4g}")
    return off, out, dx, dw


if __name__ == "__main__":
    main()
