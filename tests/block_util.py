"""Plain 64-bit forms and tolerances for the tests of a transformer block's dense parts: the product with bias,
activation and residual, the norm and rotation of heads, and their backward passes."""
import math

import torch

from ops_util import DT, U32, rounding

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
LEAST = 1e-36     # exp2 underflows below: what an activation's far tail may lose
SLOPE = 2.0 ** -17  # absolute error of a derivative: see slope_error


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return z * torch.sigmoid(_inner(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "relu":
        return torch.where(z > 0, torch.ones_like(z), torch.where(z == z, torch.zeros_like(z), z))
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        s = torch.sigmoid(_inner(z))
        return s + z * s * (1 - s) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def _inner(z):
    return math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)


def act_error(z, act):
    """What an activation in fp32 steps may be off by.  Sixteen roundings of its value (2^-20: for gelu the polynomial's
    5e-7 is eight of them, the reciprocal, exp2 and products the others), and the rounding of the exponent q, in which
    exp2's argument has up to four roundings: q * 2^-22."""
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    q = z * z / 2 if act == "gelu" else _inner(z).abs() if act == "gelu_tanh" else z.abs()
    return act64(z, act).abs() * (2.0 ** -20 + q * 2.0 ** -22) + LEAST


def linear64(a, w, bias, act, r):
    """(z, c, what z may be off by in fp32 sums, what c may be off by before its rounding).  A sum of K exact products, in any
    order, is off by at most one rounding of the terms' magnitudes each; bias and joins are six more.  No activation is steeper than 1.13."""
    a, w = a.double().cpu(), w.double().cpu()
    z, size = a @ w.t(), a.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias.double().cpu(), size + bias.double().cpu().abs()
    ez = (a.shape[1] + 6) * U32 * size
    c = act64(z, act)
    ec = 1.13 * ez + act_error(z, act)
    if r is not None:
        ec = ec + 2 * U32 * (c.abs() + r.double().cpu().abs())
        c = c + r.double().cpu()
    return z, c, ez, ec


def linear_bwd64(dc, z, a, w, act, dtype):
    """((dz, da, dw, db), what each may be off by before its rounding).

    A derivative is off by less than SLOPE: the sigmoid's error is at most s (1 - s) times its argument's (four roundings
    of q, and q s (1 - s) < 0.28) and two roundings; in d s (1 - s), d < 3 q, that gives 4 * 3 q^2 s (1 - s) < 7
    roundings, its products 6, and 1 - s, off by one rounding of 1, up to 51 (it is 0 from q = 17 on): below
    2^7 roundings of 1.  dz is rounded to `dtype` before the products read it."""
    dc, z, a, w = (t.double().cpu() if t is not None else None for t in (dc, z, a, w))
    dz = dc if act == "none" else dc * slope64(z, act)
    e = dc.abs() * (SLOPE if act not in ("none", "relu") else 0.0) + U32 * dz.abs()
    ez = e + (rounding(dz, dtype) if dtype is not None else 0.0)
    M, N = dz.shape
    mag = dz.abs() + ez
    return (dz, dz @ w, dz.t() @ a, dz.sum(0)), (e, ez @ w.abs() + (N + 6) * U32 * (mag @ w.abs()),
                                                 ez.t() @ a.abs() + (M + 6) * U32 * (mag.t() @ a.abs()),
                                                 e.sum(0) + (M + 6) * U32 * mag.sum(0))


# ------------------------------------------------------------------ heads

def turn64(v, angles, positions, pairs, back=False, size=False):
    """v (tokens x heads x dim, 64 bits) turned; size: what the terms of each element add up to in magnitude."""
    if angles is None:
        return v.abs() if size else v
    cos, sin = (t.double().cpu()[positions.cpu()][:, None] for t in angles)
    half = cos.shape[2]
    i = torch.arange(half)
    first, second = (i, i + half) if pairs == "halves" else (2 * i, 2 * i + 1)
    x, y = v[..., first], v[..., second]
    out = v.clone()
    if size:
        out = out.abs()
        out[..., first], out[..., second] = (x * cos).abs() + (y * sin).abs(), (y * cos).abs() + (x * sin).abs()
        return out
    if back:
        sin = -sin
    out[..., first], out[..., second] = x * cos - y * sin, y * cos + x * sin
    return out


STEPS = 32 + 6 + 16   # roundings on the longest way into a head's sums: a lane's elements, joins of lanes and of waves


def heads64(x, w, angles, positions, pairs, eps):
    """(y, what it may be off by before its rounding): half of a sum's roundings reach the root, then the root, the quotient,
    the products by rstd, w and the angle's, and one sum: 8."""
    x = x.double().cpu()
    v = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        v = v * w.double().cpu()
    return turn64(v, angles, positions, pairs), (STEPS / 2 + 8) * U32 * turn64(v, angles, positions, pairs, size=True)


def heads_bwd64(dy, x, w, angles, positions, pairs, eps):
    """((dx, dw), what each may be off by before its rounding).  Each of dx's terms holds rstd up to three times (half of a
    sum's roundings each), a turned gradient and w, and the mean a sum of its own: 3 * (STEPS / 2 + 4) + STEPS + 8 roundings of
    the terms' magnitudes; a term of dw half a sum's and 8, their sum one more each."""
    dy, x = dy.double().cpu(), x.double().cpu()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = x * rstd
    g = turn64(dy, angles, positions, pairs, back=True)
    big = turn64(dy, angles, positions, pairs, size=True)
    dw, dw_size = (g * u).sum((0, 1)), (big * u.abs()).sum((0, 1))
    if w is not None:
        g, big = g * w.double().cpu(), big * w.double().cpu().abs()
    dx = rstd * (g - u * (g * u).mean(-1, keepdim=True))
    size = rstd * (big + u.abs() * (big * u.abs()).mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    return (dx, dw), ((3 * (STEPS / 2 + 4) + STEPS + 8) * U32 * size, (rows + STEPS / 2 + 8) * U32 * dw_size)


def name_of(dtype):
    return next(n for n, t in DT.items() if t == dtype)
