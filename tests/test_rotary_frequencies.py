"""kvp_rotary_frequencies (host arithmetic) against exact decimal arithmetic, and what is refused
before any launch (CPU only)."""

import ctypes
from decimal import Decimal, getcontext

import pytest

from libbuild import ensure_built

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def exact_turns(dim, i, base, scaling, factor, original, low, high):
    b = Decimal(base)
    if scaling == "ntk":
        b *= Decimal(factor) ** (Decimal(dim) / Decimal(dim - 2))
    t = b ** (Decimal(-2 * i) / Decimal(dim))
    if scaling == "linear":
        t /= Decimal(factor)
    if scaling == "by_parts":
        keep = (Decimal(original) * t / (2 * PI) - Decimal(low)) / (Decimal(high) - Decimal(low))
        keep = min(Decimal(1), max(Decimal(0), keep))
        t = keep * t + (1 - keep) * t / Decimal(factor)
    return t / (2 * PI)


@pytest.mark.parametrize("dim", [2, 16, 64, 128])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("by_parts", 40.0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies_are_the_formulas(dim, scaling, factor, base):
    kb = ensure_built()
    if scaling == "ntk" and dim == 2:
        with pytest.raises(kb.KvpError):
            kb.rotary_frequencies(dim, base, scaling, factor)
        return
    got = kb.rotary_frequencies(dim, base, scaling, factor, 4096, 1.0, 32.0)
    assert len(got) == dim // 2
    for i, f in enumerate(got):
        want = exact_turns(dim, i, base, scaling, factor, 4096, 1, 32)
        # a pow, up to four more double operations (2^-53 each; pow below 2^-52), the base's own rounding amplified
        # by the exponent (ntk), then 2^-64 of a turn
        assert abs(Decimal(f) / 2 ** 64 - want) <= want * Decimal(2) ** -48 + Decimal(2) ** -64


def test_bad_frequencies_are_refused():
    kb = ensure_built()
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, base=0.0),
               dict(rotary_dim=8, base=float("nan")), dict(rotary_dim=8, scaling="linear", factor=0.0),
               dict(rotary_dim=8, scaling="linear", factor=float("inf")),
               dict(rotary_dim=8, scaling="by_parts", factor=2.0, original_len=0),
               dict(rotary_dim=8, scaling="by_parts", factor=2.0, low_turns=4.0, high_turns=4.0)):
        with pytest.raises(kb.KvpError) as e:
            kb.rotary_frequencies(**kw)
        assert e.value.code == kb.KVP_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        kb.rotary_frequencies(8, scaling="other")


def test_argument_checks_without_a_gpu():
    """Host checks that need no pool: nothing here reaches a launch."""
    kb = ensure_built()
    lib, null, p = kb.lib(), ctypes.c_void_p(), ctypes.c_void_p(256)
    BAD = kb.KVP_ERR_INVALID_ARG
    assert lib.rotary_store_cache(null, 0, p, 8, 8, 1, p, 8, p, 8, p, p, 1, p, 8, 0, 1.0, p, 8, 8, null) == BAD
    assert lib.rotary_store_latent(null, 0, p, 8, 8, 1, p, 8, p, 8, p, p, 1, p, 8, 0, 1.0, p, 8, 8, null) == BAD
    assert lib.paged_latent_attention(null, 0, p, 1, 1, 1, null, p, 1, 1, 0, null, p, 0, 0, 1.0, p, p, 256, null) == BAD
    n = ctypes.c_size_t()
    assert lib.paged_latent_attention_workspace_size(null, 1, 1, 1, ctypes.byref(n)) == BAD
    out = ctypes.c_void_p()
    for dims in ((0, 64), (512, -1), (1025, 64), (512, 1025)):
        assert lib.kv_latent_pool_create(4, 4, *dims, 1, 1, p, p, ctypes.byref(out)) == BAD
    assert lib.kv_latent_pool_create(4, 4, 512, 64, 1, 1, ctypes.c_void_p(8), p, ctypes.byref(out)) == BAD
    assert lib.kv_latent_pool_create(4, 4, 13, 2, 1, 1, p, p, ctypes.byref(out)) == BAD  # 30-byte rows

    def prefill(q=p, qs=192, qh=192, k=p, ks=128, kh=128, pe=p, ps=64, v=p, vs=128, vh=128, q0=p, k0=p, B=1, H=1, mq=4,
                tq=4, tk=4, dn=128, dr=64, dv=128, dt=1, scale=1.0, o=p):
        return lib.latent_prefill_attention(q, qs, qh, k, ks, kh, pe, ps, v, vs, vh, q0, k0, B, H, mq, tq, tk, dn, dr, dv,
                                            dt, scale, o, null, null)

    for kw in (dict(q=null), dict(k=null), dict(pe=null), dict(v=null), dict(o=null), dict(q0=null), dict(k0=null),
               dict(B=0), dict(H=0), dict(mq=-1), dict(tq=-1), dict(tk=-1), dict(dn=0), dict(dr=-1), dict(dv=0),
               dict(dn=513), dict(dr=513), dict(dv=513), dict(dt=7), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(qh=-1), dict(qs=-1), dict(kh=-1), dict(ks=-1), dict(vh=-1),
               dict(vs=-1), dict(ps=-1), dict(q=ctypes.c_void_p(257)), dict(o=ctypes.c_void_p(257))):
        assert prefill(**kw) == BAD, kw
    assert prefill(mq=0) == kb.KVP_OK and prefill(tq=0) == kb.KVP_OK  # no query: nothing is launched
