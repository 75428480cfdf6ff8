"""Plain 64-bit references of the rotary, latent and expanded operators, each
with an elementwise bound on what its arithmetic may be off by.

Roundings count ``u(dtype) = finfo.eps / 2`` relative each; U32 = 2^-24 is
that of the fp32 arithmetic inside the kernels.
"""

import math

import torch

U32 = 2.0 ** -24


def u(dtype):
    return torch.finfo(dtype).eps / 2


def thetas(dim, base=10000.0, scaling="none", factor=1.0, original=4096, low=1.0, high=32.0):
    out = []
    for i in range(dim // 2):
        b = base * (factor ** (dim / (dim - 2)) if scaling == "ntk" else 1.0)
        t = b ** (-2.0 * i / dim)
        if scaling == "linear":
            t /= factor
        if scaling == "by_parts":
            keep = min(1.0, max(0.0, (original * t / (2 * math.pi) - low) / (high - low)))
            t = keep * t + (1 - keep) * t / factor
        out.append(t)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, positions, theta, layout, attn=1.0):
    """x [n, H, D] -> (rotated float64, bound): the first 2 len(theta) entries turned."""
    x = x.double().cpu()
    dim = 2 * len(theta)
    ang = positions.double().cpu()[:, None] * theta
    c, s = ang.cos()[:, None] * attn, ang.sin()[:, None] * attn
    if layout == "half":
        ia, ib = torch.arange(0, dim // 2), torch.arange(dim // 2, dim)
    else:
        ia, ib = torch.arange(0, dim, 2), torch.arange(1, dim, 2)
    y, bound = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # the fraction of a turn is rounded to 24 bits of at most half a turn (pi * 2^-24 radians), the sine and cosine
    # to 2 units of fp32, attn and the two products and their sum to one each: below 8 U32 (|a| + |b|) attn; the
    # reference's own angle, a double, is off by 2^-53 of itself
    off = (8 * U32 + ang.abs()[:, None] * 2.0 ** -51) * (a.abs() + b.abs()) * attn
    bound[..., ia], bound[..., ib] = off, off
    return y, bound


def span(p, window, sinks):
    """Positions that the query at position p attends."""
    if window <= 0:
        return list(range(p + 1))
    lo = max(0, p + 1 - (window - sinks))
    return list(range(min(sinks, lo))) + list(range(lo, p + 1))


def attend(q, keys, values, scale, dtype):
    """q [H, W], keys [n, W] or [n, H, W], values likewise, float64 -> (out [H, dv], bound).

    A score is an fp32 sum of W exact products: off by at most W U32 sum |q x| scale, and the scaling, the shift by
    the maximum and the exponential add 2^-21 of the scores' size. That error e moves a weight by e relative, and the
    sum of weights as much. Under bf16 each weight is rounded once more (u) before it meets its value. The sums over
    n values are off by n U32 at most; the result is rounded once (u)."""
    H, W = q.shape
    if keys.dim() == 2:
        keys = keys[:, None].expand(-1, H, -1)
    if values.dim() == 2:
        values = values[:, None].expand(-1, H, -1)
    s = torch.einsum("hw,nhw->hn", q, keys) * scale
    mag = torch.einsum("hw,nhw->hn", q.abs(), keys.abs()) * abs(scale)
    e = ((W + 4) * U32 * mag + 2.0 ** -21 * (s.abs() + s.abs().amax(-1, keepdim=True))).amax(-1)
    w = torch.softmax(s, -1)
    out = torch.einsum("hn,nhd->hd", w, values)
    wabs = torch.einsum("hn,nhd->hd", w, values.abs())
    n = keys.shape[0]
    rel = 2 * torch.expm1(e) + 2 * (n + 16) * U32 + (2 * u(dtype) if dtype == torch.bfloat16 else 0.0)
    return out, rel[:, None] * wabs + u(dtype) * out.abs() + 1e-30


def check(got, want, bound, what=""):
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} entries off, worst "
                           f"{float((d / bound.clamp(min=1e-300)).nan_to_num(float('inf')).max()):.3g} x its bound")
