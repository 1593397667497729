"""Heads whose strides' products pass 64 bits: refused as any heads that overlap, or that no memory holds."""
import pytest

from test_block_cpu import P, heads, no_gpu, qk, qk_bwd, refused

HUGE = [
    (1 << 30, 3, 1 << 39, 1 << 38),             # token 1 lies between heads 2 and 4; (tokens - 1) * ld passes 2^63
    ((1 << 30) - 1, 2, (1 << 39) + 40, 1 << 37),
    (1 << 25, 3, 1 << 39, 1 << 38),             # passes 2^63 by one bit
    (1 << 30, 65536, 1 << 39, 1 << 23),         # no overlap, but no memory holds it
    (1 << 30, 1, (1 << 40) - 1, 0),
]


@no_gpu
@pytest.mark.parametrize("tokens,n,ld,hs", HUGE)
def test_heads_past_64_bits_are_refused(tokens, n, ld, hs):
    far, near = heads(ld, hs), heads(n * 40, 40, P)
    base = dict(tokens=tokens, q_heads=n, k_heads=0, rope=None)
    refused(qk(q=far, out_q=near, **base))
    refused(qk(q=near, out_q=far, **base))
    for name in ("dq", "q", "dxq"):
        refused(qk_bwd(**{**dict(dq=near, q=near, dxq=near), name: far}, **base))
