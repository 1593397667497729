"""One transformer block through libgemm's operators for its dense parts, trained and served.

    y = rmsnorm(x)                                                        (gemm_rmsnorm)
    qkv = y Wqkv^T + bias                                                 (gemm_linear)
    q, k = norm of each head, turned by the token's position              (gemm_qk_norm_rope)
    x = attention(q, k, v) Wo^T + x                                       (gemm_linear; the attention itself in plain torch)
    x = gelu(rmsnorm(x) Wup^T + bias) Wdown^T + x                         (gemm_rmsnorm, gemm_linear twice)
Training: a step's gradients through autograd (the backward passes of all three).
Serving: the prompt at once, then single tokens with a cache of keys and values.  Needs one GPU:
    python examples/dense_block.py [--width 4096] [--wide 14336] [--heads 32] [--groups 8] [--prompt 512] [--tokens 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tiled_stage_software_amd import ops  # noqa: E402


def attention(q, k, v, first=0):
    """Causal attention of tokens first, first + 1, ... (q) over tokens 0, 1, ... (k, v), in fp32."""
    each = q.shape[1] // k.shape[1]
    q, k, v = (t.float().transpose(0, 1).contiguous() for t in (q, k, v))
    k, v = (t.repeat_interleave(each, 0) for t in (k, v))
    score = q @ k.transpose(1, 2).contiguous() / q.shape[2] ** 0.5
    at, to = torch.arange(k.shape[1], device=q.device), first + torch.arange(q.shape[1], device=q.device)
    p = score.masked_fill(at > to[:, None], float("-inf")).softmax(2)
    return (p @ v).transpose(0, 1).flatten(1)


class Block:
    def __init__(self, width, wide, heads, groups, tokens, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.groups, self.dim = heads, groups, width // heads
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        weight = lambda n, k: (randn(n, k) / k ** 0.5).bfloat16().requires_grad_()  # noqa: E731
        scale = lambda n: (1 + 0.1 * randn(n)).bfloat16().requires_grad_()  # noqa: E731
        out = (heads + 2 * groups) * self.dim
        self.parameters = dict(norm1=scale(width), qkv=weight(out, width), qkv_bias=(0.1 * randn(out)).bfloat16().requires_grad_(),
                               q_norm=scale(self.dim), k_norm=scale(self.dim), proj=weight(width, heads * self.dim), norm2=scale(width),
                               up=weight(wide, width), up_bias=(0.1 * randn(wide)).bfloat16().requires_grad_(), down=weight(width, wide))
        self.cos, self.sin = ops.rope_table(tokens, self.dim, device="cuda")

    def forward(self, x, positions, cache=None):
        """x: tokens x width; with a cache (keys, values of all tokens), x's are written to it at `positions`."""
        p = self.parameters
        qkv = ops.linear(ops.rmsnorm(x, p["norm1"]).y, p["qkv"], p["qkv_bias"]).unflatten(1, (-1, self.dim))
        q, k, v = qkv.split([self.heads, self.groups, self.groups], 1)
        q, k = ops.qk_norm_rope(q, k, p["q_norm"], p["k_norm"], positions, self.cos, self.sin)
        first = 0
        if cache is not None:
            first = int(positions[0])
            for held, new in zip(cache, (k, v)):
                held[first:first + len(x)] = new
            k, v = (held[:first + len(x)] for held in cache)
        x = ops.linear(attention(q, k, v, first).to(x.dtype), p["proj"], residual=x)
        up = ops.linear(ops.rmsnorm(x, p["norm2"]).y, p["up"], p["up_bias"], act="gelu")
        return ops.linear(up, p["down"], residual=x)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--wide", type=int, default=14336)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args(argv)
    total = a.prompt + a.tokens
    block = Block(a.width, a.wide, a.heads, a.groups, total)
    positions = torch.arange(total, device="cuda")

    # a training step's gradients
    x = torch.randn(total, a.width, device="cuda").bfloat16().requires_grad_()
    for _ in range(2):
        torch.cuda.synchronize()
        start = time.perf_counter()
        out = block.forward(x, positions)
        dy = torch.randn(out.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
        of = torch.autograd.grad(out, [x, *block.parameters.values()], dy)
        torch.cuda.synchronize()
    print(f"step of {total} tokens: {(time.perf_counter() - start) * 1e3:.2f} ms")

    # the same tokens served: the prompt, then one by one
    with torch.no_grad():
        cache = [torch.zeros(total, a.groups, block.dim, dtype=x.dtype, device="cuda") for _ in range(2)]
        served = [block.forward(x[:a.prompt], positions[:a.prompt], cache)]
        torch.cuda.synchronize()
        start = time.perf_counter()
        for t in range(a.prompt, total):
            served.append(block.forward(x[t:t + 1], positions[t:t + 1], cache))
        torch.cuda.synchronize()
    if a.tokens:
        print(f"{a.tokens} tokens: {(time.perf_counter() - start) / a.tokens * 1e6:.0f} us each")
    return block, x, dy, out.detach(), torch.cat(served), dict(zip(["x", *block.parameters], of))


if __name__ == "__main__":
    main()
