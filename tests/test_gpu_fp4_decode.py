"""The decode kernel of four-bit pools at its edges. Contexts are bounded above 256 rows, where short ones go to the tile
kernel, unless a case is about both."""

import math

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from test_gpu_fp4_attention import DEV, Case, kb  # noqa: F401

pytestmark = pytest.mark.gpu
LOG2E = math.log2(math.e)
FAR = 1000  # a bound of the lengths that keeps few short contexts with the decode kernel


def bounded(c, most, fill=0x3C):
    c.most = most
    c.ws = c.kb.alloc_fp4_workspace(c.pool, len(c.lens), c.C, c.H, most, device=DEV)
    c.ws.fill_(fill)
    return c


def rewrite(c, k, v):
    """Every request's rows: the first of k, v [L, D], the same for every head."""
    each = lambda x: x.to(c.dt).to(DEV)[:, None].expand(-1, c.hkv, -1).contiguous()  # noqa: E731
    for sl in c.slots:
        c.kb.store_cache_fp4(c.pool, c.layer, each(k[:len(sl)]), each(v[:len(sl)]), torch.tensor(sl, dtype=torch.int32, device=DEV))
    c.read()


def scale_for(factor):
    """A scale whose product with log2(e) is ``factor`` (a power of two) in fp32."""
    log2e = torch.tensor(LOG2E, dtype=torch.float32)
    s = torch.tensor(factor / LOG2E, dtype=torch.float32)
    for step in (0.0, math.inf, -math.inf):
        x = s if step == 0.0 else torch.nextafter(s, torch.tensor(step))
        if float(x * log2e) == factor:
            return float(x)
    raise AssertionError("no such scale")


@pytest.mark.parametrize("C,raw", [(1, False), (4, False), (1, True)])
def test_scores_a_step_of_fp32_apart(kb, C, raw):  # noqa: F811
    """Scores about 2^27 in log2, where fp32's step is 16: the maximum rises by one step from a stage of 32 rows to the
    next. A row 16 below the maximum weighs 2^-16."""
    L = 320  # of so many requests that a piece of the work is several stages
    c = bounded(Case(kb, "bf16", [L] * 200, C, 8, 8, 128, 1 if raw else 16, raw, seed=1), FAR)
    k, v = torch.zeros(L, 128), torch.randn(L, 128, generator=torch.Generator().manual_seed(2))
    k[:, 0] = k[:, 1] = 1024.0
    k[:, 16] = 2.0 ** -4
    k[:, 15], k[:, 31] = 6 * 256.0, 6 * 2.0 ** -3  # these only make the blocks' scales 256 and 2^-3
    k[160:, 16] = 2.0 ** -3  # q . k is 2048 + 2^-12 in the first 160 rows, then 2048 + 2^-11
    rewrite(c, k, v)
    assert torch.equal(c.k[c.slots[0], 0], k.double())
    c.q.zero_()
    c.q[..., 0] = c.q[..., 1] = 1.0
    c.q[..., 16] = 2.0 ** -8
    c.scale = scale_for(2.0 ** 16)
    c.run()
    out, vals = c.out.double().cpu(), c.v[c.slots[0], 0]
    for j in range(C):
        s = torch.where(torch.arange(L) < 160, 0.0, 16.0)[:L - C + j + 1]
        w = torch.exp2(s - 16)
        want = (w[:, None] * vals[:len(w)]).sum(0) / w.sum()
        # the weights are powers of two: what is left is the fp32 sums and the result's rounding
        bound = R.u(torch.bfloat16) * want.abs() + 2 * (len(w) + 16) * R.U32 * vals.abs().amax(0)
        R.check(out[:, j], want.expand(200, 8, -1), bound.expand(200, 8, -1), f"query {j}")


@pytest.mark.parametrize("C,at", [(1, 0), (1, 1500), (1, 2999), (4, 0), (4, 1500)])
@pytest.mark.parametrize("gap", [26.5, 30.0])
def test_many_rows_far_below_one(kb, C, at, gap):  # noqa: F811
    """One row far above thousands that weigh 2^-gap each and alone have values: they are the result, whether the one
    comes first, in the middle or last."""
    L, B = 3000, 40
    c = Case(kb, "bf16", [L] * B, C, 8, 2, 128, 16, seed=1)
    k, v = torch.zeros(L, 128), torch.rand(L, 128, generator=torch.Generator().manual_seed(2)) + 0.5
    k[:, 0], k[at, 0], v[at] = 1.0, 6.0, 0.0
    rewrite(c, k, v)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.scale = gap / 5 / LOG2E
    c.run()
    for j in range(C):
        p = L - C + j
        sl = torch.tensor(c.slots[0][:p + 1])
        want, bound = F.attend(c.q[0, j, :1].double().cpu(), c.k[sl, 0], c.v[sl, 0], c.scale, c.dt)
        # a weight is off by half a step of fp16, or, below 2^-14 of a largest one that is 2^7 at least, by 2^-32 of that
        bound = bound + (2.0 ** -32 - 2.0 ** -25) * (p + 1) * c.v[sl, 0].abs().amax()
        R.check(c.out[:, j].cpu(), want.expand(B, 8, -1), bound.expand(B, 8, -1), f"query {j}")


@pytest.mark.parametrize("C,raw,sign", [(1, False, 1), (1, False, -1), (1, True, 1), (4, False, 1), (4, True, -1), (20, False, 1)])
def test_scores_that_rise_stage_by_stage(kb, C, raw, sign):  # noqa: F811
    """Every 32 rows score 10 above the 32 before in log2: the maximum is raised with each, in both directions of time."""
    L = 32 * 63 - 5
    c = Case(kb, "bf16", [L] * 20 + [33], C, 8, 8, 128, 1 if raw else 16, raw, seed=1)
    g = torch.Generator().manual_seed(2)
    k, v = torch.zeros(L, 128), torch.randn(L, 128, generator=g)
    at = torch.arange(L) // 32
    for i in range(6):
        k[:, 16 * i] = torch.where(at >> i & 1 > 0, 2.0 ** i, 0.0)
    rewrite(c, k, v)
    c.q.zero_()
    c.q[..., ::16] = float(sign)
    c.scale = 10 / LOG2E
    c.run()
    c.verify(only=[0, 7, 19, 20], few=True)


@pytest.mark.parametrize("most", [250, 257, FAR])
@pytest.mark.parametrize("C,H,hkv", [(1, 32, 8), (4, 32, 8), (1, 32, 16), (2, 4, 1)])
@pytest.mark.parametrize("times,fill", [(1, 0x00), (1, 0x3C), (60, 0x00), (200, 0x3C)])
def test_bad_requests_are_zeros_and_recorded(kb, C, H, hkv, times, fill, most):  # noqa: F811
    """Invalid requests among few, whose pieces are recorded by request, and among many, by CTA; in workspaces of zeros and
    of small numbers."""
    lens = [200, 4, 220, 170, 250] * times
    c = bounded(Case(kb, "bf16", lens, C, H, hkv, 128, 16, seed=6), most, fill)
    clens, rows = torch.tensor(lens), torch.arange(5 * times)
    clens[1::5], clens[2::5], rows[3::5] = 0, 100000, 5 * times + 7
    clens[3::15] = -3
    c.clens.copy_(clens)
    c.run(table_rows=rows.to(torch.int32).to(DEV))
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    for i in (1, 2, 3):
        assert bool((c.out[i::5] == 0).all()), i
    last = 5 * times
    c.verify(only=sorted({0, 4, last - 5, last - 1}))


@pytest.mark.parametrize("C,raw,P", [(1, False, 16), (4, False, 16), (1, False, 4), (1, True, 16), (4, True, 1), (20, True, 1)])
def test_holes_are_skipped_and_recorded(kb, C, raw, P):  # noqa: F811
    """Holes, entries past the pool and far past it, in pages that come whole and in rows that come one by one."""
    c = bounded(Case(kb, "bf16", [200, 220, 300], C, 32, 8, 128, P, raw, seed=6), FAR)
    c.table[0, 3] = -1
    c.table[0, 5] = 1 << 30
    c.table[0, 11] = c.pool.num_pages * (P if raw else 1)
    c.table[2] = -1
    c.run()
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    c.verify(only=[1])


@pytest.mark.parametrize("C,raw", [(1, False), (4, False), (1, True)])
def test_queries_of_any_size(kb, C, raw):  # noqa: F811
    c = bounded(Case(kb, "bf16", [150, 99, 400], C, 32, 8, 128, 1 if raw else 16, raw, seed=9), FAR)
    for h, e in ((0, -100), (1, -40), (3, 100), (6, -126)):
        c.q[:, :, h] *= 2.0 ** e
    c.q[:, :, 4] = 0
    c.q[:, :, 5, ::3] *= 2.0 ** -30
    c.run()
    out = c.out.cpu()
    assert not bool(out.isnan().any())
    for b in range(3):
        for j in range(C):
            w, bound = c.want(b, j, C)
            keep = [h for h in range(32) if h != 3]
            R.check(out[b, j, keep], w[keep], bound[keep])
            R.check(out[b, j, 3], w[3], R.u(torch.bfloat16) * w[3].abs() + 1e-30)  # one key has all the weight


@pytest.mark.parametrize("C", [1, 4])
def test_queries_that_are_not_finite(kb, C):  # noqa: F811
    c = bounded(Case(kb, "bf16", [150, 700], C, 32, 8, 128, 16, seed=9), FAR)
    c.q[0, 0, 3, 7] = float("nan")
    c.q[1, C - 1, 9, 7] = float("inf")
    c.run()
    bad = c.out.isnan().all(-1).cpu()
    assert bool(bad[0, 0, 3]) and bool(bad[1, C - 1, 9]) and int(c.out.isnan().any(-1).sum()) == 2
    for b, j, h in ((0, 0, 3), (1, C - 1, 9)):
        w, bound = c.want(b, j, C)
        keep = [x for x in range(32) if x != h]
        R.check(c.out[b, j, keep].cpu(), w[keep], bound[keep])


@pytest.mark.parametrize("C,H,hkv", [(1, 32, 8), (4, 32, 8), (1, 8, 2)])
def test_groups_together_and_apart_in_turn(kb, C, H, hkv):  # noqa: F811
    """A raw table whose groups of 16 rows lie together (one copy) and apart (row by row) by turns of odd length, so that a
    buffer's scales come now by the one and now by the other kind of copy; the same bits each time."""
    c = Case(kb, "bf16", [1500 + i for i in range(40)], C, H, hkv, 128, 16, raw=True, seed=4)
    g = torch.Generator().manual_seed(5)
    table = c.table.cpu()
    for b, sl in enumerate(c.slots):
        for t in range(0, len(sl) - 16, 16):
            if (t // 16) % 7 in (2, 3, 5):
                sl[t:t + 16] = [sl[t + i] for i in torch.randperm(16, generator=g).tolist()]
        table[b, :len(sl)] = torch.tensor(sl)
    c.table.copy_(table)
    first = c.run().clone()
    c.verify(only=[0, 13, 39])
    for _ in range(5):
        c.run()
        assert torch.equal(first, c.out)
