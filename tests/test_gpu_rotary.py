"""rotary_store_cache and rotary_store_latent against the 64-bit formulas."""

import pytest
import torch

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


def make(kb, dtype, n, Hq, Hkv, D, P, seed, layers=1):
    g = torch.Generator().manual_seed(seed)
    pages = -(-n // P) + 2
    kv = torch.full((2, layers, pages, P, Hkv, D), 7.0, dtype=DT[dtype], device=DEV)
    pool = kb.Pool(kv, P, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32)
    loc = torch.randperm(pages * P, generator=g)[:n].to(torch.int32)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g).to(DT[dtype]).to(DEV)
    return pool, kv, loc, qkv


def expect(qkv, Hq, Hkv, pos, theta, layout, attn, dt):
    q, qb = R.rotate(qkv[:, :Hq], pos, theta, layout, attn)
    k, kbnd = R.rotate(qkv[:, Hq:Hq + Hkv], pos, theta, layout, attn)
    return q, qb + R.u(dt) * (q.abs() + qb), k, kbnd + R.u(dt) * (k.abs() + kbnd)


CASES = [
    # dtype, n, Hq, Hkv, D, rot, P, layout, scaling, factor, far
    ("bf16", 1, 32, 8, 128, 128, 16, "half", "none", 1.0, 1),
    ("bf16", 64, 32, 8, 128, 128, 16, "half", "by_parts", 8.0, 100000),
    ("bf16", 333, 16, 2, 128, 64, 1, "interleaved", "linear", 4.0, 1 << 20),
    ("bf16", 5000, 8, 2, 64, 64, 16, "half", "ntk", 2.0, 4096),          # several tokens a block
    ("bf16", 5001, 4, 4, 64, 32, 4, "interleaved", "none", 1.0, 70000),  # and a short last block
    ("bf16", 17, 4, 2, 128, 0, 16, "half", "none", 1.0, 99),             # nothing turns
    ("bf16", 9, 3, 1, 80, 40, 4, "half", "none", 1.0, 5000),             # rot / 2 = 20: element by element
    ("bf16", 9, 3, 1, 72, 24, 4, "interleaved", "none", 1.0, 5000),      # a rest of 48 entries
    ("bf16", 6, 2, 2, 12, 6, 4, "half", "none", 1.0, 5000),              # head rows of 24 bytes
    ("bf16", 31, 40, 8, 128, 128, 16, "half", "none", 1.0, 5000),
    ("f32", 3001, 16, 2, 64, 64, 4, "interleaved", "ntk", 2.0, 32768),
    ("f32", 100, 2, 2, 16, 16, 4, "half", "none", 1.0, 1 << 20),
    ("f32", 7, 2, 2, 20, 10, 4, "half", "none", 1.0, 300),
    ("f32", 50, 5, 1, 512, 512, 16, "half", "none", 1.0, 300),
    ("f32", 50, 5, 1, 2048, 1024, 16, "half", "none", 1.0, 300),         # one token's pairs fill the block's table
    ("f32", 5, 2, 1, 2048, 2048, 16, "interleaved", "none", 1.0, 300),   # and do not fit it
]


@pytest.mark.parametrize("dtype,n,Hq,Hkv,D,rot,P,layout,scaling,factor,far", CASES)
def test_rotary_store_is_the_formula(kb, dtype, n, Hq, Hkv, D, rot, P, layout, scaling, factor, far):
    pool, kv, loc, qkv = make(kb, dtype, n, Hq, Hkv, D, P, seed=n)
    before = kv.clone()
    attn = 1.25 if scaling == "by_parts" else 1.0
    pos = torch.randint(0, far, (n,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    if rot:
        rope = kb.RotaryPlan(rot, layout=layout, scaling=scaling, factor=factor, attn_factor=attn, device=DEV)
    else:
        rope = kb.RotaryPlan(2, layout=layout, device=DEV)
        rope.rotary_dim = 0
    q_out = torch.full((n, Hq, D), float("nan"), dtype=DT[dtype], device=DEV)
    kb.rotary_store_cache(pool, 0, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos.to(DEV), loc.to(DEV), rope, q_out)
    q, qb, k, kbd = expect(qkv, Hq, Hkv, pos, R.thetas(rot, scaling=scaling, factor=factor), layout, attn, DT[dtype])
    R.check(q_out, q, qb, "q")
    rows = kv.view(2, -1, Hkv, D)
    R.check(rows[0, loc.long()], k, kbd, "k")
    assert torch.equal(rows[1, loc.long()], qkv[:, Hq + Hkv:]), "v must be copied as it is"
    # no other row of the pool changed
    keep = torch.ones(rows.shape[1], dtype=torch.bool)
    keep[loc.long()] = False
    assert torch.equal(rows[:, keep.to(DEV)], before.view(2, -1, Hkv, D)[:, keep.to(DEV)])
    assert kb.kvp_sync_error(pool) == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_to_the_ends_of_int32(kb, layout):
    """The largest and most negative positions: the fixed-point fraction loses nothing, so the bound only
    grows by the 2^-53 that theta / 2 pi is off by, times the position, in turns."""
    pool, kv, loc, qkv = make(kb, "f32", 6, 2, 1, 64, 4, seed=8)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, -123456789], dtype=torch.int32)
    rope = kb.RotaryPlan(64, layout=layout, device=DEV)
    q_out = torch.empty((6, 2, 64), device=DEV)
    kb.rotary_store_cache(pool, 0, qkv[:, :2], qkv[:, 2:3], qkv[:, 3:], pos.to(DEV), loc.to(DEV), rope, q_out)
    theta = R.thetas(64)
    q, qb = R.rotate(qkv[:, :2], pos, theta, layout)
    R.check(q_out, q, qb + R.U32 * q.abs(), "q")
    assert torch.equal(q_out[0], qkv[0, :2]), "position 0 turns nothing"


def test_in_place_and_parts(kb):
    """q in place over a view of the projection; only q; only the store."""
    n, Hq, Hkv, D = 40, 8, 2, 128
    pool, kv, loc, qkv = make(kb, "bf16", n, Hq, Hkv, D, 16, seed=4)
    pos = torch.arange(100, 100 + n, dtype=torch.int32, device=DEV)
    rope = kb.RotaryPlan(D, device=DEV)
    loc = loc.to(DEV)
    want = torch.empty((n, Hq, D), dtype=torch.bfloat16, device=DEV)
    src = qkv.clone()
    kb.rotary_store_cache(pool, 0, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, loc, rope, want)
    kept = kv.clone()
    assert torch.equal(qkv, src), "the inputs stay as they were"
    kv.fill_(7.0)
    kb.rotary_store_cache(pool, 0, None, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, loc, rope, None)
    assert torch.equal(kv, kept)
    kv.fill_(7.0)
    only = torch.empty_like(want)
    kb.rotary_store_cache(pool, 0, qkv[:, :Hq], None, None, pos, None, rope, only)
    assert torch.equal(only, want) and bool((kv == 7.0).all())
    kb.rotary_store_cache(pool, 0, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, loc, rope, qkv[:, :Hq])
    assert torch.equal(qkv[:, :Hq], want) and torch.equal(qkv[:, Hq:], src[:, Hq:]) and torch.equal(kv, kept)


def test_odd_strides_and_alignment(kb):
    """Rows that start on odd elements take the element-wise kernel, with the same results."""
    n, Hq, Hkv, D = 13, 4, 2, 64
    pool, kv, loc, qkv = make(kb, "bf16", n, Hq, Hkv, D, 4, seed=5)
    wide = torch.zeros((n, (Hq + 2 * Hkv) * D + 7), dtype=torch.bfloat16, device=DEV)
    wide[:, 3:3 + qkv[0].numel()] = qkv.flatten(1)
    view = wide[:, 3:3 + qkv[0].numel()].unflatten(1, (Hq + 2 * Hkv, D))
    pos = torch.arange(n, dtype=torch.int32, device=DEV) * 1000
    for layout in ("half", "interleaved"):
        rope = kb.RotaryPlan(D, layout=layout, device=DEV)
        outs = []
        for t in (qkv, view):
            kv.zero_()
            o = torch.empty((n, Hq, D), dtype=torch.bfloat16, device=DEV)
            kb.rotary_store_cache(pool, 0, t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], pos, loc.to(DEV), rope, o)
            outs.append((o, kv.clone()))
        q, qb, _, _ = expect(qkv, Hq, Hkv, pos, R.thetas(D), layout, 1.0, torch.bfloat16)
        for o, _ in outs:
            R.check(o, q, qb, layout)


def test_bad_slots_are_skipped(kb):
    n, Hq, Hkv, D = 8, 4, 2, 64
    for D, name in ((64, "vector"), (12, "element")):
        pool, kv, loc, qkv = make(kb, "bf16", n, Hq, Hkv, D, 4, seed=6)
        good = loc.clone()
        loc[2], loc[5] = -1, pool.num_pages * pool.page_size
        rope = kb.RotaryPlan(4 if D == 12 else D, device=DEV)
        q_out = torch.empty((n, Hq, D), dtype=torch.bfloat16, device=DEV)
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        kb.rotary_store_cache(pool, 0, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, loc.to(DEV), rope, q_out)
        assert kb.kvp_sync_error(pool) == kb.KVP_ERR_BAD_INDEX
        rows = kv.view(2, -1, Hkv, D)
        for i in range(n):
            if i in (2, 5):
                assert bool((rows[:, good[i].item()] == 7.0).all()), name
            else:
                assert torch.equal(rows[1, good[i].item()], qkv[i, Hq + Hkv:]), name
        q, qb, _, _ = expect(qkv, Hq, Hkv, pos, R.thetas(rope.rotary_dim), "half", 1.0, torch.bfloat16)
        R.check(q_out, q, qb, name)


def test_second_layer_other_stream_and_graph(kb):
    n, Hq, Hkv, D = 70, 8, 2, 128
    pool, kv, loc, qkv = make(kb, "bf16", n, Hq, Hkv, D, 16, seed=7, layers=3)
    loc = loc.to(DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    rope = kb.RotaryPlan(D, device=DEV)
    q_out = torch.empty((n, Hq, D), dtype=torch.bfloat16, device=DEV)
    call = lambda **kw: kb.rotary_store_cache(pool, 1, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, loc,  # noqa: E731
                                              rope, q_out, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    s.synchronize()
    assert bool((kv[:, 0] == 7.0).all()) and bool((kv[:, 2] == 7.0).all())
    first, q1 = kv.clone(), q_out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    kv.fill_(7.0)
    q_out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kv, first) and torch.equal(q_out, q1)
    pos += 5  # the graph reads the buffers it was given
    g.replay()
    torch.cuda.synchronize()
    q, qb, _, _ = expect(qkv, Hq, Hkv, pos, R.thetas(D), "half", 1.0, torch.bfloat16)
    R.check(q_out, q, qb, "replay")


LATENT = [
    # dtype, n, Hq, dc, dr, P, layout
    ("bf16", 1, 16, 512, 64, 16, "interleaved"),
    ("bf16", 256, 16, 512, 64, 16, "interleaved"),
    ("bf16", 777, 128, 512, 64, 64, "half"),
    ("bf16", 6000, 8, 512, 64, 1, "half"),
    ("bf16", 20, 3, 100, 12, 4, "half"),   # element by element
    ("f32", 99, 4, 128, 32, 4, "half"),
    ("f32", 9, 4, 6, 2, 4, "interleaved"),
]


@pytest.mark.parametrize("dtype,n,Hq,dc,dr,P,layout", LATENT)
def test_latent_store_is_the_formula(kb, dtype, n, Hq, dc, dr, P, layout):
    g = torch.Generator().manual_seed(n)
    dt = DT[dtype]
    pages = -(-n // P) + 2
    buf = torch.full((2, pages, P, dc + dr), 7.0, dtype=dt, device=DEV)
    pool = kb.LatentPool(buf, dc, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32)
    loc = torch.randperm(pages * P, generator=g)[:n]
    down = torch.randn((n, dc + dr), generator=g).to(dt).to(DEV)
    q_pe = torch.randn((n, Hq, dr), generator=g).to(dt).to(DEV)
    q = torch.full((n, Hq, dc + dr), 3.0, dtype=dt, device=DEV)
    pos = torch.randint(0, 200000, (n,), generator=g).to(torch.int32)
    rope = kb.RotaryPlan(dr, layout=layout, scaling="by_parts", factor=40.0, attn_factor=1.37, device=DEV)
    kb.rotary_store_latent(pool, 1, q_pe, down[:, :dc], down[:, dc:], pos.to(DEV), loc.to(torch.int32).to(DEV), rope,
                           q[..., dc:])
    theta = R.thetas(dr, scaling="by_parts", factor=40.0)
    wq, bq = R.rotate(q_pe, pos, theta, layout, rope.attn_factor)
    wk, bk = R.rotate(down[:, None, dc:], pos, theta, layout, rope.attn_factor)
    R.check(q[..., dc:], wq, bq + R.u(dt) * (wq.abs() + bq), "q_pe")
    assert bool((q[..., :dc] == 3.0).all())
    rows = buf[1].view(-1, dc + dr)
    assert torch.equal(rows[loc.to(DEV), :dc], down[:, :dc])
    R.check(rows[loc.to(DEV)][:, None, dc:], wk, bk + R.u(dt) * (wk.abs() + bk), "k_pe")
    rest = torch.ones(rows.shape[0], dtype=torch.bool)
    rest[loc] = False
    assert bool((rows[rest.to(DEV)] == 7.0).all()) and bool((buf[0] == 7.0).all())
    assert kb.kvp_sync_error(pool) == 0


@pytest.mark.parametrize("dtype,dc", [("bf16", 512), ("bf16", 8), ("f32", 20), ("bf16", 1024)])
def test_latent_rows_without_a_rotated_part(kb, dtype, dc):
    """rope_dim 0: only the latents are stored, queries and key parts have no entries."""
    g = torch.Generator().manual_seed(dc)
    buf = torch.full((2, 40, 4, dc), 7.0, dtype=DT[dtype], device=DEV)
    pool = kb.LatentPool(buf, dc, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32)
    n, none = 33, torch.empty((33, 0), dtype=DT[dtype], device=DEV)
    lat = torch.randn((n, 2 * dc), generator=g).to(DT[dtype]).to(DEV)[:, :dc]
    loc = torch.randperm(160, generator=g)[:n].to(torch.int32)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    rope = kb.RotaryPlan(0, device=DEV)
    kb.rotary_store_latent(pool, 1, None, lat, none, pos, loc.to(DEV), rope, None)
    kb.rotary_store_latent(pool, 0, none[:, None].expand(n, 3, 0), lat, none, pos, loc.to(DEV), rope,
                           torch.empty((n, 3, 0), dtype=DT[dtype], device=DEV))
    want = torch.full((160, dc), 7.0, dtype=DT[dtype])
    want[loc.long()] = lat.cpu()
    for layer in range(2):
        assert torch.equal(buf[layer].view(160, dc).cpu(), want)
    assert kb.kvp_sync_error(pool) == 0


def test_slots_past_four_gigabytes(kb):
    Hkv, D, P, slots, n = 8, 128, 16, 2_200_000, 40
    kv = torch.empty((2, 1, slots // P, P, Hkv, D), dtype=torch.bfloat16, device=DEV)
    pool = kb.Pool(kv, P, kb.KVP_BF16)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((n, Hkv, D), generator=g).bfloat16().to(DEV) for _ in range(2))
    loc = (slots - 1 - torch.randperm(500, generator=g)[:n]).to(torch.int32).to(DEV)
    kb.rotary_store_cache(pool, 0, None, k, v, torch.zeros(n, dtype=torch.int32, device=DEV), loc,
                          kb.RotaryPlan(D, device=DEV), None)
    for plane, want in ((kv[0, 0], k), (kv[1, 0], v)):
        assert torch.equal(plane.view(slots, Hkv, D)[loc.long()], want)
    assert kb.kvp_sync_error(pool) == 0


def test_refusals(kb):
    pool, kv, loc, qkv = make(kb, "bf16", 8, 4, 2, 64, 4, seed=1)
    rope = kb.RotaryPlan(64, device=DEV)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    pos, loc = torch.zeros(8, dtype=torch.int32, device=DEV), loc.to(DEV)
    out = torch.empty((8, 4, 64), dtype=torch.bfloat16, device=DEV)
    call = kb.rotary_store_cache
    with pytest.raises(TypeError):
        call(pool, 0, q.float(), k, v, pos, loc, rope, out)
    with pytest.raises(TypeError):
        call(pool, 0, q, k, v, pos.long(), loc, rope, out)
    with pytest.raises(ValueError):
        call(pool, 0, q[:7], k, v, pos, loc, rope, out)
    with pytest.raises(ValueError):
        call(pool, 0, q, k, None, pos, loc, rope, out)
    with pytest.raises(ValueError):
        call(pool, 0, None, None, None, pos, loc, rope, None)
    with pytest.raises(ValueError):
        call(pool, 0, q, k, v, pos, loc, kb.RotaryPlan(128, device=DEV), out)
    with pytest.raises(ValueError):
        call(pool, 0, q, k.transpose(0, 1).contiguous().transpose(0, 1), v, pos, loc, rope, out)  # heads apart
    with pytest.raises(ValueError):
        call(pool, 0, q[..., ::2], k, v, pos, loc, rope, out)
    for layer in (-1, 1):
        with pytest.raises(kb.KvpError):
            call(pool, layer, q, k, v, pos, loc, rope, out)
    latents = kb.LatentPool(torch.zeros((1, 4, 4, 64), dtype=torch.bfloat16, device=DEV), 48, kb.KVP_BF16)
    with pytest.raises((kb.KvpError, ValueError)):
        call(latents, 0, q, k, v, pos, loc, rope, out)
    # the calls of K/V pools refuse a latent pool, whatever the binding lets through
    L, p = kb.lib(), kb._ptr(kv)
    BAD = kb.KVP_ERR_INVALID_ARG
    h = latents.handle
    assert L.store_cache(h, 0, p, p, p, 1, None) == BAD
    assert L.paged_decode_attention(h, 0, p, 1, 1, p, 1, 1, 0, None, p, 0, 0, 1.0, p, p, 1 << 30, None) == BAD
    assert L.paged_prefill_attention(h, 0, p, 1, 1, 1, None, p, 1, 1, 0, None, p, 0, 0, 1.0, p, None) == BAD
    assert L.rotary_store_cache(h, 0, p, 64, 64, 1, None, 0, None, 0, p, None, 1, p, 64, 0, 1.0, p, 64, 64, None) == BAD
    assert L.rotary_store_latent(pool.handle, 0, p, 64, 64, 1, None, 0, None, 0, p, None, 1, p, 64, 0, 1.0, p, 64, 64,
                                 None) == BAD
    # q over itself with other strides would read what it has written
    assert L.rotary_store_cache(pool.handle, 0, p, 256, 64, 4, None, 0, None, 0, p, None, 1, p, 64, 0, 1.0, p, 512, 64,
                                None) == BAD
    call(pool, 0, q[:0], k[:0], v[:0], pos[:0], loc[:0], rope, out[:0])  # nothing to do
    torch.cuda.synchronize()
    assert kb.kvp_sync_error(pool) == 0


@pytest.mark.parametrize("layout,D", [("half", 64), ("interleaved", 64), ("half", 12)])
def test_sines_and_cosines_keep_their_bits(kb, layout, D):
    """The turned pair (1, 0) is (cos, sin). With a turn's quadrant taken off exactly, what is left of the angle, t with
    |t| <= pi / 4, is rounded to fp32 once (U32 |t|; the bits below 2^-34 of a turn, 0.006 U32, are cut), and sincospif is
    within one unit in the last place (2 U32 of the value). With |t| <= 1.12 |sin t| the sine of it is off by (3.12 |sin t|
    + 0.007) U32, the cosine by (0.57 + 2 |cos t|) U32 <= 2.9 |cos t| U32. 355, 710 and the like lie next to multiples of pi."""
    import math
    from fractions import Fraction

    pos = [0, 1, 2, 3, 11, 22, 33, 44, 88, 355, 710, 1065, 51819, 52174, 103993, 104348, 1000003, 2 ** 31 - 1, -355, -2 ** 31]
    n, rot = len(pos), D
    buf = torch.zeros((2, 1, 8, 4, 1, D), device=DEV)
    pool = kb.Pool(buf, 4, kb.KVP_F32)
    rope = kb.RotaryPlan(rot, layout=layout, device=DEV)
    first = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    q = torch.zeros((n, 1, D), device=DEV)
    q[..., first] = 1.0
    out = torch.empty_like(q)
    kb.rotary_store_cache(pool, 0, q, None, None, torch.tensor(pos, dtype=torch.int32, device=DEV), None, rope, out)
    want_c, want_s = torch.empty((n, rot // 2), dtype=torch.float64), torch.empty((n, rot // 2), dtype=torch.float64)
    for x, p in enumerate(pos):
        for i, f in enumerate(kb.rotary_frequencies(rot)):
            t = p * f % (1 << 64)
            k = (t + (1 << 61)) >> 62  # the nearest quarter turn
            a = 2 * math.pi * float(Fraction(t - (k << 62), 1 << 64))
            c, s = math.cos(a), math.sin(a)
            want_c[x, i], want_s[x, i] = ((c, s), (-s, c), (-c, -s), (s, -c))[k % 4]
    for got, want in ((out[:, 0, first], want_c), (out[:, 0, second], want_s)):
        R.check(got, want, R.U32 * (3.2 * want.abs() + 0.01), layout)


def test_as_many_tokens_as_int32_counts(kb):
    """Queries alone, in place: 2^31 - 1 tokens of one head of 8 entries (34 GB), all at the same position but the ends."""
    n, D = 2 ** 31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free memory")
    pool = kb.Pool(torch.zeros((2, 1, 2, 4, 1, D), dtype=torch.bfloat16, device=DEV), 4, kb.KVP_BF16)
    q = torch.ones((n, 1, D), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(n, dtype=torch.int32, device=DEV)
    ends = torch.tensor([0, 1, 2, n // 2, n - 3, n - 2, n - 1], device=DEV)
    pos[ends] = torch.arange(1, 8, dtype=torch.int32, device=DEV) * 1000
    kb.rotary_store_cache(pool, 0, q, None, None, pos, None, kb.RotaryPlan(D, layout="interleaved", device=DEV), q)
    want, bound = R.rotate(torch.ones((7, 1, D)), pos[ends].cpu(), R.thetas(D), "interleaved")
    R.check(q[ends], want, bound + R.u(torch.bfloat16) * (want.abs() + bound), "ends")
    assert int((pos != 0).sum()) == 7
    for at in range(3, n - 3, 1 << 28):  # the rest stays: position 0 turns nothing
        part = q[at:min(at + (1 << 28), n - 3)]
        moved = int((part != 1).any(-1).sum())
        assert moved == (1 if at <= n // 2 < at + (1 << 28) else 0)
    assert kb.kvp_sync_error(pool) == 0
