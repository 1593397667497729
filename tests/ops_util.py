"""Inputs, plain 64-bit forms and tolerances for the tests of the operators around the products."""
import torch

U32 = 2.0 ** -24        # half a step of fp32, relative
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
SMALLEST = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25,
            torch.float8_e4m3fn: 2.0 ** -10}  # half the least step


def padded(values, pad, dev, fill=0x7F, lead=0):
    """A device view of `values` whose rows lie `pad` elements further apart, `lead` elements
    into its memory; every byte around them is `fill`.  Returns (view, whole buffer)."""
    rows, cols = values.shape
    es = values.element_size()
    buf = torch.full(((rows * (cols + pad) + lead + 8) * es,), fill, dtype=torch.uint8, device=dev)
    whole = buf.view(values.dtype)
    view = whole[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(values.to(dev))
    return view, whole


def untouched(view, whole, fill=0x7F):
    """Whether every byte of `whole` outside `view` still is `fill`."""
    mask = torch.ones(whole.numel(), dtype=torch.bool, device=whole.device)
    lead = (view.data_ptr() - whole.data_ptr()) // whole.element_size()
    rows, cols = view.shape
    at = lead + torch.arange(rows, device=whole.device)[:, None] * view.stride(0) + torch.arange(cols, device=whole.device)
    mask[at.reshape(-1)] = False
    return bool((whole.view(torch.uint8).view(-1, whole.element_size())[mask] == fill).all())


def off(got, want, allowed):
    """The largest error over what is allowed (non-finite values have to agree)."""
    got, want, allowed = got.double().cpu(), want.double().cpu(), allowed.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(want), torch.isnan(got)), "NaN in other places"
    assert torch.equal(want[~fine & ~torch.isnan(want)], got[~fine & ~torch.isnan(want)]), "infinities differ"
    if not bool(fine.any()):
        return 0.0
    return float(((got - want).abs() / allowed)[fine].max())


def rounding(want, dtype):
    """Half a step of `dtype` at `want`."""
    return want.abs() * (torch.finfo(dtype).eps / 2) + SMALLEST[dtype]


# ------------------------------------------------------------------ norm

def norm64(x, r, w, eps):
    """(h as kept, rstd, y) in 64 bits."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    v = h.double()
    rstd = 1 / torch.sqrt((v * v).mean(1) + eps)
    y = v * rstd[:, None]
    return h, rstd, y if w is None else y * w.double()


def norm_steps(cols):
    """Roundings on the longest way into a row's sum: a thread's own elements (at most 32, or
    every 1024th where the row is looped over), 6 joins of lanes, up to 16 of waves."""
    return max(32, cols // 1024 + 8) + 6 + 16


def norm_bwd64(dy, h, w, rstd, dh):
    """(dx, dw, what dx's terms add up to in magnitude, the same of dw)"""
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    u = h * rstd
    g = dy if w is None else dy * w.double()
    dx = rstd * (g - u * (g * u).mean(1, keepdim=True))
    size = rstd.abs() * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return dx, (dy * u).sum(0), size, (dy * u).abs().sum(0)


# ------------------------------------------------------------------ products

def f8_64(a, b, sa, sb):
    """(the product, the sum of its terms' magnitudes)"""
    a, b = a.double().cpu(), b.double().cpu()
    if sa is not None:
        a = a * sa.double().cpu()[:, None]
    if sb is not None:
        b = b * sb.double().cpu()[:, None]
    return a @ b.t(), a.abs() @ b.abs().t()


def f8_cut(a, b, sa, sb):
    """What the 8-bit matrix instructions may cut off a 16-bit C: of each eight consecutive k
    the products but the largest lose less than 2^-13 of it each."""
    k = -(-a.shape[1] // 8) * 8
    wide = lambda t, s: torch.nn.functional.pad((t.float() if s is None else t.float() * s[:, None]).abs(),  # noqa: E731
                                                (0, k - t.shape[1])).view(t.shape[0], k // 8, 8)
    a, b = wide(a, sa), wide(b, sb)
    out = torch.empty(a.shape[0], b.shape[0], dtype=torch.float64)
    for m in range(a.shape[0]):
        out[m] = (a[m][None] * b).amax(2).double().sum(1)
    return out * (7 * 2.0 ** -13)


def unpack4(codes, k):
    codes = codes.cpu()
    return torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :k]


def w4_64(a, codes, scales, zeros, group):
    """(the product, the magnitude that its rounding errors go by: each group's
    16 |s| sum |a| (2 + 1 + |z|/16), the terms the kernel adds)"""
    a = a.double().cpu()
    k = a.shape[1]
    each = lambda t: t.double().cpu().repeat_interleave(group, 1)[:, :k]  # noqa: E731
    s = each(scales)
    z = torch.full_like(s, 8.0) if zeros is None else each(zeros)
    w = s * (unpack4(codes, k).double() - z)
    return a @ w.t(), a.abs() @ (16 * s.abs() * (3 + z.abs() / 16)).t()
