"""The store into a four-bit pool, the rows read back and page copies, against the 64-bit formulas: codes and scales are
equal, not near."""

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


def make_pool(kb, pages, P, hkv, D, dtype, layers=1, ks=1.0, vs=1.0):
    pool = kb.kv_fp4_pool_create(pages, P, hkv, D, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32, layers, ks, vs, device=DEV)
    pool.codes.fill_(0xAB)
    pool.scales.fill_(0xCD)
    return pool


def slots_of(n, total, g):
    return torch.randperm(total, generator=g)[:n].to(torch.int32)


def check_rows(pool, loc, want_k, want_v, gk, gv, layer=0):
    codes, scales = F.unpack(pool, layer)
    for part, want, g in ((0, want_k, gk), (1, want_v, gv)):
        wc, ws = F.quantise(want, g)
        assert torch.equal(scales[loc.long(), :, part], ws), "scales"
        assert F.same_codes(codes[loc.long(), :, part], wc), "codes"
    rest = torch.ones(codes.shape[0], dtype=torch.bool)
    rest[loc.long()] = False
    assert bool((codes[rest] == torch.tensor([0xB, 0xA]).repeat(codes.shape[-1] // 2)).all()), "rows of other slots"
    assert bool((scales[rest] == 0xCD).all()), "scales of other slots"


STORES = [
    # dtype, n, hq, hkv, D, rot, P, layout, sections, interleave
    ("bf16", 1, 32, 8, 128, 128, 16, "half", None, False),
    ("bf16", 67, 32, 8, 128, 128, 16, "half", None, False),
    ("bf16", 67, 8, 2, 128, 128, 16, "interleaved", None, False),
    ("bf16", 67, 8, 8, 128, 64, 1, "half", None, False),
    ("bf16", 67, 8, 1, 128, 64, 4, "interleaved", (8, 12, 12), True),
    ("bf16", 67, 4, 4, 64, 64, 16, "half", (16, 8, 8), False),
    ("bf16", 67, 4, 4, 64, 32, 3, "half", None, False),
    ("bf16", 67, 4, 4, 64, 16, 16, "half", None, False),         # half of a block turned: block by block
    ("bf16", 67, 4, 4, 64, 6, 16, "interleaved", (1, 1, 1), False),
    ("bf16", 67, 8, 8, 16, 16, 16, "half", None, False),
    ("bf16", 67, 8, 8, 16, 16, 16, "interleaved", None, False),
    ("bf16", 67, 2, 2, 256, 256, 16, "half", (43, 43, 42), True),
    ("bf16", 67, 8, 8, 48, 32, 16, "half", None, False),
    ("bf16", 9000, 8, 2, 128, 128, 16, "half", (24, 20, 20), True),  # four tokens a block
    ("f32", 67, 8, 2, 128, 128, 16, "half", None, False),
    ("f32", 67, 8, 2, 64, 32, 16, "interleaved", (4, 6, 6), False),
    ("f32", 67, 8, 2, 64, 10, 16, "half", None, False),
    ("f32", 9000, 2, 2, 64, 64, 1, "half", None, False),
]


@pytest.mark.parametrize("dtype,n,hq,hkv,D,rot,P,layout,sections,interleave", STORES)
def test_store_is_the_formula(kb, dtype, n, hq, hkv, D, rot, P, layout, sections, interleave):
    g = torch.Generator().manual_seed(n + D + rot)
    pages = -(-n // P) + 3
    gk, gv = 2.0, 0.25
    pool = make_pool(kb, pages, P, hkv, D, dtype, layers=2, ks=[1.0, gk], vs=[4.0, gv])
    qkv = torch.randn((n, hq + 2 * hkv, D), generator=g).to(DT[dtype])
    loc = slots_of(n, pages * P, g)
    axes = len(sections) if sections else 1
    pos = torch.randint(-(1 << 20), 1 << 20, (axes, n), generator=g, dtype=torch.int32)
    plan = kb.RotaryPlan(rot, layout=layout, attn_factor=1.25, device=DEV, sections=sections, interleave=interleave)
    d = qkv.to(DEV)
    q, k, v = d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:]
    q_out = torch.zeros((n, hq, D), dtype=DT[dtype], device=DEV)
    kb.rotary_store_fp4(pool, 1, q, k, v, (pos if axes > 1 else pos[0]).to(DEV), loc.to(DEV), plan, q_out)
    torch.cuda.synchronize()
    assert kb.kvp_sync_error(pool) == 0
    theta = R.thetas(rot)
    of_pair = kb.pair_axes(sections, interleave) if sections else [0] * (rot // 2)
    wq, bound = F.rotate_axes(qkv[:, :hq], pos, theta, of_pair, layout, 1.25)
    R.check(q_out, wq, bound + R.u(DT[dtype]) * (wq.abs() + bound), "q")
    wk, _ = F.rotate_axes(qkv[:, hq:hq + hkv], pos, theta, of_pair, layout, 1.25)
    check_rows(pool, loc, wk, qkv[:, hq + hkv:].double(), gk, gv, layer=1)
    assert bool((pool.codes[0] == 0xAB).all()) and bool((pool.scales[0] == 0xCD).all()), "the other layer"
    # read back, any order, twice the same slot
    back = torch.cat((loc.flip(0), loc[:1])).to(DEV)
    ko, vo = (torch.empty((n + 1, hkv, D), dtype=DT[dtype], device=DEV) for _ in range(2))
    kb.load_cache_fp4(pool, 1, back, ko, vo)
    codes, scales = F.unpack(pool, 1)
    for part, got, gs in ((0, ko, gk), (1, vo, gv)):
        want = F.values(codes[back.cpu().long(), :, part], scales[back.cpu().long(), :, part], gs)
        assert torch.equal(got.double().cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("aligned", [True, False])
def test_borders_and_extremes(kb, dtype, aligned):
    """Values on and next to every border of codes and scales, blocks of zeros, tiny, huge and not finite ones; rows that
    start on 16 bytes, and rows that do not."""
    g = torch.Generator().manual_seed(5)
    hkv, D, n = 8, 64, 64
    mant = torch.randint(8, 16, (n, 2 * hkv, D // 16, 1), generator=g).double()
    expo = torch.randint(-12, 13, (n, 2 * hkv, D // 16, 1), generator=g).double()
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[torch.randint(0, 8, (n, 2 * hkv, D // 16, 16),
                                                                                     generator=g)].double()
    x = border * mant * torch.exp2(expo)
    x[..., 0] = 6 * (mant * torch.exp2(expo))[..., 0]  # the scale is mant * 2^expo
    if dtype == "f32":  # one step of fp32 beside the border
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, x, torch.nextafter(x.float(), torch.rand(
            x.shape, generator=g) * 100 - 50).double())
    x = x * torch.where(torch.rand(x.shape, generator=g) < 0.5, 1.0, -1.0)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 2.0 ** -20      # scales below e4m3's smallest normal one
    x[3] *= 2.0 ** -60      # and that round to zero
    x[4] *= 2.0 ** 40       # saturate
    x[5, :, 0, 3] = float("inf")
    x[6, :, 1, 4] = float("nan")
    x[7, :, :, 5] = float("-inf")
    # the midpoints of two scales, and one step beside them
    x[8:24] = torch.rand((16, 2 * hkv, D // 16, 16), generator=g).double()
    x[8:24, ..., 7] = 6 * (2 * mant[8:24, ..., 0] + 1) * torch.exp2(expo[8:24, ..., 0].clamp(-8, 4)) / 2 ** 3
    x[24:28] = x[8:12]
    x[24:28, ..., 7] *= 1 + 2.0 ** -7
    if dtype == "f32":
        x[28:32] = x[8:12]
        x[28:32, ..., 7] *= 1 - 2.0 ** -24
    x = x.flatten(-2).to(DT[dtype])
    pool = make_pool(kb, 8, 16, hkv, D, dtype)
    buf = torch.zeros(n * 2 * hkv * D + 1, dtype=DT[dtype], device=DEV)
    kv = buf[0 if aligned else 1:][:n * 2 * hkv * D].view(n, 2 * hkv, D)
    kv.copy_(x)
    loc = slots_of(n, 128, g)
    kb.store_cache_fp4(pool, 0, kv[:, :hkv], kv[:, hkv:], loc.to(DEV))
    assert kb.kvp_sync_error(pool) == 0
    check_rows(pool, loc, x[:, :hkv].double(), x[:, hkv:].double(), 1.0, 1.0)
    ko, vo = (torch.empty((n, hkv, D), dtype=DT[dtype], device=DEV) for _ in range(2))
    kb.load_cache_fp4(pool, 0, loc.to(DEV), ko, vo)
    assert bool(ko[5:7, :, :32].isnan().any(-1).all()) and bool(ko[7].isnan().all()) and not bool(ko[8:].isnan().any())


@pytest.mark.parametrize("e", [-64, 64])
def test_global_scales_at_their_ends(kb, e):
    """g = 2^-64 and 2^64: the codes of the values over g; far values saturate, with their signs."""
    g = torch.Generator().manual_seed(11)
    n, hkv, D = 20, 2, 64
    x = torch.randn((n, 2 * hkv, D), generator=g).to(torch.bfloat16).double() * 2.0 ** e
    x[3] *= 2.0 ** 30
    x[4, :, ::2] = -3e38 if e < 0 else 2.0 ** 100
    pool = make_pool(kb, 4, 16, hkv, D, "bf16", ks=2.0 ** e, vs=2.0 ** e)
    loc = slots_of(n, 64, g)
    d = x.to(torch.bfloat16).to(DEV)
    kb.store_cache_fp4(pool, 0, d[:, :hkv], d[:, hkv:], loc.to(DEV))
    x = d.double().cpu()
    check_rows(pool, loc, x[:, :hkv], x[:, hkv:], 2.0 ** e, 2.0 ** e)


def test_rows_as_they_are_at_position_zero(kb):
    """Nothing turns at position zero: borders are met exactly, where only 64 bits decide."""
    g = torch.Generator().manual_seed(6)
    n, hkv, D = 40, 4, 64
    x = (torch.randint(-40, 41, (n, 2 * hkv, D), generator=g).double() / 8).to(torch.bfloat16)
    pool = make_pool(kb, 4, 16, hkv, D, "bf16")
    loc = slots_of(n, 64, g)
    d = x.to(DEV)
    kb.rotary_store_fp4(pool, 0, None, d[:, :hkv], d[:, hkv:], torch.zeros(n, dtype=torch.int32, device=DEV), loc.to(DEV),
                        kb.RotaryPlan(D, device=DEV), None)
    check_rows(pool, loc, x[:, :hkv].double(), x[:, hkv:].double(), 1.0, 1.0)


def test_bad_slots_are_skipped(kb):
    g = torch.Generator().manual_seed(7)
    n, hkv, D = 33, 2, 64
    pool = make_pool(kb, 4, 16, hkv, D, "bf16")
    loc = slots_of(n, 64, g)
    loc[3], loc[20] = -1, 64
    x = torch.randn((n, 2 * hkv, D), generator=g).to(torch.bfloat16)
    d = x.to(DEV)
    for kv in (d, torch.cat((torch.zeros(1, dtype=d.dtype, device=DEV), d.flatten()))[1:].view(d.shape)):
        pool.codes.fill_(0xAB)
        pool.scales.fill_(0xCD)
        kb.store_cache_fp4(pool, 0, kv[:, :hkv], kv[:, hkv:], loc.to(DEV))
        assert kb.kvp_sync_error(pool) == kb.KVP_ERR_BAD_INDEX
        good = (loc >= 0) & (loc < 64)
        check_rows(pool, loc[good], x[good, :hkv].double(), x[good, hkv:].double(), 1.0, 1.0)
    ko, vo = (torch.full((n, hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kb.load_cache_fp4(pool, 0, loc.to(DEV), ko, vo)
    assert kb.kvp_sync_error(pool) == kb.KVP_ERR_BAD_INDEX
    assert bool((ko[[3, 20]] == 0).all()) and bool((vo[[3, 20]] == 0).all()) and bool((ko[good.to(DEV)] != 7.0).all())


def test_nothing_to_do(kb):
    pool = make_pool(kb, 4, 16, 2, 64, "bf16")
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    kb.store_cache_fp4(pool, 0, e, e, none)
    kb.load_cache_fp4(pool, 0, none, e, e)
    kb.rotary_store_fp4(pool, 0, e, e, e, none, none, kb.RotaryPlan(64, device=DEV), e)
    assert bool((pool.codes == 0xAB).all())


def test_queries_alone_and_in_place(kb):
    g = torch.Generator().manual_seed(8)
    pool = make_pool(kb, 4, 16, 2, 64, "bf16")
    x = torch.randn((21, 5, 64), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 4096, (3, 21), generator=g, dtype=torch.int32)
    plan = kb.RotaryPlan(64, device=DEV, sections=(16, 8, 8))
    q = x.to(DEV)
    kb.rotary_store_fp4(pool, 0, q, None, None, pos.to(DEV), None, plan, q)
    w, bound = F.rotate_axes(x, pos, R.thetas(64), kb.pair_axes((16, 8, 8)), "half")
    R.check(q, w, bound + R.u(torch.bfloat16) * (w.abs() + bound))
    assert bool((pool.codes == 0xAB).all())


@pytest.mark.parametrize("P,D,hkv", [(16, 128, 8), (1, 128, 1), (5, 64, 2), (24, 48, 8)])
def test_pages_are_copied_whole(kb, P, D, hkv):
    g = torch.Generator().manual_seed(9)
    pool = make_pool(kb, 9, P, hkv, D, "bf16", layers=3)
    pool.codes.copy_(torch.randint(0, 256, pool.codes.shape, generator=g, dtype=torch.uint8))
    pool.scales.copy_(torch.randint(0, 127, pool.scales.shape, generator=g, dtype=torch.uint8))
    for dev_count in (False, True):
        before = [F.unpack(pool, layer) for layer in range(3)]
        src, dst = torch.tensor([0, 4, 4, 99], dtype=torch.int32), torch.tensor([8, 1, 7, 3], dtype=torch.int32)
        m = 3 if dev_count else 4
        if dev_count:
            kb.copy_pages_device_count(pool, src.to(DEV), dst.to(DEV), torch.tensor([3], dtype=torch.int32, device=DEV))
        else:
            kb.copy_pages(pool, src.to(DEV), dst.to(DEV))
        assert kb.kvp_sync_error(pool) == (0 if dev_count else kb.KVP_ERR_BAD_INDEX)
        for layer in range(3):
            for b, a in zip(before[layer], F.unpack(pool, layer)):
                want = b.clone().view(9, P, *b.shape[1:])
                for s, t in zip(src.tolist()[:min(m, 3)], dst.tolist()):
                    want[t] = b.view(want.shape)[s]
                assert torch.equal(a, want.view(a.shape))


def test_rows_past_four_gigabytes(kb):
    """Codes and scales of slots whose byte offsets pass 32 bits."""
    hkv, D, P = 8, 128, 16
    pages = (1 << 32) // (hkv * D * P) + 300
    pool = kb.kv_fp4_pool_create(pages, P, hkv, D, kb.KVP_BF16, 2, device=DEV)
    g = torch.Generator().manual_seed(10)
    n = 40
    loc = (pages * P - 1 - torch.arange(n) * 7).to(torch.int32)
    x = torch.randn((n, 2 * hkv, D), generator=g).to(torch.bfloat16)
    d = x.to(DEV)
    kb.store_cache_fp4(pool, 1, d[:, :hkv], d[:, hkv:], loc.to(DEV))
    ko, vo = (torch.empty((n, hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kb.load_cache_fp4(pool, 1, loc.to(DEV), ko, vo)
    assert kb.kvp_sync_error(pool) == 0
    for got, want in ((ko, x[:, :hkv]), (vo, x[:, hkv:])):
        c, s = F.quantise(want.double(), 1.0)
        assert torch.equal(got.double().cpu(), F.values(c, s, 1.0))
    src = torch.tensor([pages - 1], dtype=torch.int32, device=DEV)
    kb.copy_pages(pool, src, torch.tensor([0], dtype=torch.int32, device=DEV))
    assert torch.equal(pool.codes[1, 0], pool.codes[1, -1])
    assert torch.equal(pool.scales[1, 0], pool.scales[1, pages * P // 16 - 1])
