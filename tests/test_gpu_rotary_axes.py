"""Rotary positions of several axes on K/V and latent pools against the 64-bit formulas."""

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from libbuild import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_built()


CASES = [
    # dtype, n, hq, hkv, D, rot, layout, sections, interleave
    ("bf16", 1, 32, 8, 128, 128, "half", (16, 24, 24), False),
    ("bf16", 61, 32, 8, 128, 128, "half", (24, 20, 20), True),
    ("bf16", 61, 8, 2, 128, 64, "interleaved", (8, 12, 12), False),
    ("bf16", 61, 8, 2, 64, 64, "half", (0, 32), False),
    ("bf16", 61, 8, 2, 64, 24, "half", (4, 4, 4), True),      # element by element
    ("bf16", 9100, 8, 2, 128, 128, "half", (16, 24, 24), False),
    ("f32", 61, 8, 2, 64, 64, "interleaved", (4,) * 8, True),
    ("f32", 61, 8, 2, 64, 6, "interleaved", (1, 1, 1), False),
    ("f32", 9100, 4, 2, 64, 64, "interleaved", (16, 16), False),
]


@pytest.mark.parametrize("per_axis", [False, True])
@pytest.mark.parametrize("dtype,n,hq,hkv,D,rot,layout,sections,interleave", CASES)
def test_store_of_several_axes(kb, dtype, n, hq, hkv, D, rot, layout, sections, interleave, per_axis):
    g = torch.Generator().manual_seed(n + rot)
    P, pages = 16, -(-n // 16) + 2
    x = torch.randn((n, hq + 2 * hkv, D), generator=g).to(DT[dtype])
    cache = torch.full((2, 1, pages, P, hkv, D), 3.0, dtype=DT[dtype], device=DEV)
    pool = kb.Pool(cache, P, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32)
    loc = torch.randperm(pages * P, generator=g)[:n].to(torch.int32)
    wide = torch.randint(-(1 << 20), 1 << 20, (len(sections), n + 5), generator=g, dtype=torch.int32)
    pos = wide.to(DEV)[:, 2:2 + n]  # rows that lie apart
    plan = kb.RotaryPlan(rot, layout=layout, attn_factor=0.75, device=DEV, sections=sections, interleave=interleave,
                         per_axis=per_axis)
    d = x.to(DEV)
    out = torch.zeros((n, hq, D), dtype=DT[dtype], device=DEV)
    kb.rotary_store_cache(pool, 0, d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:], pos, loc.to(DEV), plan, out)
    assert kb.kvp_sync_error(pool) == 0
    of_pair = kb.pair_axes(sections, interleave)
    if per_axis:
        own = {a: iter(R.thetas(2 * of_pair.count(a))) for a in set(of_pair)}
        theta = torch.stack([next(own[a]) for a in of_pair])
    else:
        theta = R.thetas(rot)
    for got, part in ((out, x[:, :hq]), (cache.view(2, -1, hkv, D)[0, loc.to(DEV).long()], x[:, hq:hq + hkv])):
        w, bound = F.rotate_axes(part, wide[:, 2:2 + n], theta, of_pair, layout, 0.75)
        R.check(got, w, bound + R.u(DT[dtype]) * (w.abs() + bound))
    assert torch.equal(cache.view(2, -1, hkv, D)[1, loc.to(DEV).long()], d[:, hq + hkv:])


def test_equal_axes_are_one_axis(kb):
    """Text: the bits of a plan of one axis."""
    g = torch.Generator().manual_seed(2)
    n, hq, hkv, D = 50, 8, 2, 128
    x = torch.randn((n, hq + 2 * hkv, D), generator=g).to(torch.bfloat16).to(DEV)
    loc = torch.randperm(64, generator=g)[:n].to(torch.int32).to(DEV)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).to(DEV)
    got = []
    for plan, p in ((kb.RotaryPlan(D, device=DEV), pos),
                    (kb.RotaryPlan(D, device=DEV, sections=(16, 24, 24)), pos.expand(3, n).contiguous())):
        cache = torch.zeros((2, 1, 4, 16, hkv, D), dtype=torch.bfloat16, device=DEV)
        out = torch.empty((n, hq, D), dtype=torch.bfloat16, device=DEV)
        kb.rotary_store_cache(kb.Pool(cache, 16, kb.KVP_BF16), 0, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], p, loc, plan,
                              out)
        got.append((cache, out))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_latent_rows_of_several_axes(kb):
    g = torch.Generator().manual_seed(3)
    n, H, dc, dr = 45, 4, 64, 32
    buf = torch.zeros((1, 4, 16, dc + dr), dtype=torch.bfloat16, device=DEV)
    pool = kb.LatentPool(buf, dc, kb.KVP_BF16)
    down = torch.randn((n, dc + dr), generator=g).to(torch.bfloat16)
    qp = torch.randn((n, H, dr), generator=g).to(torch.bfloat16)
    loc = torch.randperm(64, generator=g)[:n].to(torch.int32)
    pos = torch.randint(0, 4096, (2, n), generator=g, dtype=torch.int32)
    q = torch.zeros((n, H, dc + dr), dtype=torch.bfloat16, device=DEV)
    d = down.to(DEV)
    kb.rotary_store_latent(pool, 0, qp.to(DEV), d[:, :dc], d[:, dc:], pos.to(DEV), loc.to(DEV),
                           kb.RotaryPlan(dr, device=DEV, sections=(4, 12)), q[..., dc:])
    of_pair = kb.pair_axes((4, 12))
    for got, part in ((q[..., dc:], qp), (buf.view(-1, dc + dr)[loc.to(DEV).long()][:, None, dc:], down[:, None, dc:])):
        w, bound = F.rotate_axes(part, pos, R.thetas(dr), of_pair, "half")
        R.check(got, w, bound + R.u(torch.bfloat16) * (w.abs() + bound))
    assert torch.equal(buf.view(-1, dc + dr)[loc.to(DEV).long()][:, :dc], d[:, :dc])


def test_an_axis_that_is_none_is_recorded(kb):
    cache = torch.zeros((2, 1, 2, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    pool = kb.Pool(cache, 16, kb.KVP_BF16)
    plan = kb.RotaryPlan(64, device=DEV, sections=(16, 16))
    plan.pair_axis[5] = 2
    x = torch.randn((3, 2, 64), device=DEV).to(torch.bfloat16)
    pos = torch.ones((2, 3), dtype=torch.int32, device=DEV)
    kb.rotary_store_cache(pool, 0, None, x, x, pos, torch.arange(3, dtype=torch.int32, device=DEV), plan, None)
    assert kb.kvp_sync_error(pool) == kb.KVP_ERR_BAD_INDEX


@pytest.mark.parametrize("page_size", [1, 16])
def test_steps_of_a_latent_cache_on_several_axes(kb, page_size):
    """Text has the same position on every axis: a step with such a plan is the one of a single axis."""
    from paged_decode_attention_store_gb300.engine import PagedLatentCache

    dc, dr, H, C = 64, 32, 4, 3
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    steps = [(rnd(2, C, H, dc + dr), rnd(2, C, H, dr), rnd(2 * C, dc), rnd(2 * C, dr)) for _ in range(3)]
    outs = []
    for sections in (None, (6, 5, 5)):
        cache = PagedLatentCache(num_pages=64, page_size=page_size, latent_dim=dc, rope_dim=dr, num_layers=1, dtype="bf16",
                                 max_requests=4, max_seq_len=64, device=DEV)
        plan = kb.RotaryPlan(dr, device=DEV, sections=sections, interleave=True)
        for rid in (0, 1):
            cache.new(rid)
        got = []
        for q, q_pe, latent, k_pe in steps:
            out = torch.empty(2, C, H, dc, dtype=torch.bfloat16, device=DEV)
            cache.step([0, 1], [q.clone()], [q_pe], [latent], [k_pe], plan, [out], window=0, scale=0.1)
            got.append(out)
        torch.cuda.synchronize()
        cache.check()
        outs.append(torch.stack(got))
    assert bool(torch.isfinite(outs[0].float()).all()) and torch.equal(outs[0], outs[1])
