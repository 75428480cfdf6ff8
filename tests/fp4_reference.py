"""Plain 64-bit references of the four-bit pool's operators and of rotary positions of several axes, with elementwise
bounds where arithmetic may be off (roundings as in operator_reference)."""

import torch

import operator_reference as R

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def nearest(x, values):
    """Index of the nearest of the ascending values, ties to the even index."""
    lo = (torch.searchsorted(values, x.contiguous(), right=True) - 1).clamp(min=0)
    hi = (lo + 1).clamp(max=len(values) - 1)
    below, above = x - values[lo], values[hi] - x
    return torch.where((hi > lo) & ((above < below) | ((above == below) & (hi % 2 == 0))), hi, lo)


def quantise(x, g):
    """x [..., D] float64 -> (codes 0 .. 15 [..., D], scale codes [..., D / 16]); blocks that are not finite: 0, 0x7f."""
    y = x.unflatten(-1, (-1, 16))
    m = y.abs().amax(-1)
    good = torch.isfinite(y).all(-1)
    m = torch.where(good, m, 0.0)
    sc = nearest(m / (6 * g), E4M3)
    s = E4M3[sc][..., None] * g
    r = torch.where((s > 0) & good[..., None], y.abs() / torch.where(s > 0, s, 1.0), 0.0)
    codes = nearest(r, E2M1) | ((y < 0) & good[..., None] & (s > 0)).long() * 8
    return codes.flatten(-2), torch.where(good, sc, 0x7f)


def values(codes, scales, g):
    """codes [..., D], scale codes [..., D / 16] -> the values they stand for, float64."""
    v = E2M1[(codes & 7).long()] * torch.where((codes & 8) > 0, -1.0, 1.0)
    s = torch.where(scales == 0x7f, float("nan"), E4M3[scales.clamp(max=126).long()]) * g
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def unpack(pool, layer=0):
    """A pool's codes [slots, Hkv, 2, D] and scale codes [slots, Hkv, 2, D / 16] on the host."""
    slots = pool.num_pages * pool.page_size
    b = pool.codes[layer].cpu().view(slots, pool.kv_heads, 2, pool.head_dim // 2).long()
    codes = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    s = pool.scales[layer].cpu().transpose(1, 2).reshape(-1, pool.kv_heads, 2, pool.head_dim // 16)[:slots].long()
    return codes, s


def same_codes(a, b):
    """Equal but for the sign of zero."""
    return bool(((a == b) | (((a & 7) == 0) & ((b & 7) == 0))).all())


def rotate_axes(x, positions, theta, of_pair, layout, attn=1.0):
    """rotate of operator_reference with positions [axes, n]: each axis' pairs by themselves."""
    half = len(theta)
    y, bound = x.double().cpu().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for a in sorted(set(of_pair)):
        ya, ba = R.rotate(x, positions[a], theta, layout, attn)
        for i in [i for i, b in enumerate(of_pair) if b == a]:
            for e in ((i, i + half) if layout == "half" else (2 * i, 2 * i + 1)):
                y[..., e], bound[..., e] = ya[..., e], ba[..., e]
    return y, bound


def attend(q, keys, vals, scale, dtype, weights=torch.float16):
    """q [H, W], keys, vals [n, W] float64 -> (out [H, W], bound): operator_reference.attend with fp16 operands.
    ``weights``: what bf16 pools' softmax weights are rounded to; the chunk kernel's are bf16, as those of a bf16 pool.

    Beyond the fp32 sums and exponentials: a query is scaled by a power of two to at most 1 and held in fp16, exact but
    below 2^-14, where it is off by 2^-25 at most: that times the keys' sizes moves a score. A weight is rounded once to
    fp16 (2^-11 relative; below 2^-14 of a maximum that is one at least, 2^-25 of it)."""
    H, W = q.shape
    s = torch.einsum("hw,nw->hn", q, keys) * scale
    mag = torch.einsum("hw,nw->hn", q.abs(), keys.abs()) * abs(scale)
    low = 2.0 ** -24 * q.abs().amax(-1)[:, None] * keys.abs().sum(-1)[None] * abs(scale)
    e = ((W + 4) * R.U32 * mag + low + 2.0 ** -21 * (s.abs() + s.abs().amax(-1, keepdim=True))).amax(-1)
    w = torch.softmax(s, -1)
    out = torch.einsum("hn,nd->hd", w, vals)
    wabs = torch.einsum("hn,nd->hd", w, vals.abs())
    n = keys.shape[0]
    half = dtype == torch.bfloat16
    rel = 2 * torch.expm1(e) + 2 * (n + 16) * R.U32 + (2 * R.u(weights) if half else 0.0)
    tiny = 2.0 ** -25 * n * vals.abs().amax() if half else 0.0
    return out, rel[:, None] * wabs + R.u(dtype) * out.abs() + tiny + 1e-30
