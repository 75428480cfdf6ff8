"""paged_latent_attention against the 64-bit formulas."""

import math

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


class Case:
    """Requests of the given lengths on shuffled pages; every slot that holds no token is NaN."""

    def __init__(self, kb, dtype, lens, C, H, dc, dr, P, raw=False, seed=0, layers=1, layer=0, spare=3, mag=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kb, self.dt, self.lens, self.C, self.H, self.dc, self.W, self.P, self.raw = (kb, DT[dtype], list(lens), C, H, dc,
                                                                                          dc + dr, P, raw)
        need = [-(-max(L, 1) // P) for L in lens]
        pages = sum(need) + spare
        self.buf = torch.full((layers, pages, P, self.W), float("nan"), dtype=self.dt)
        order = torch.randperm(pages, generator=g).tolist()
        B, cols = len(lens), max(need) + 1
        table = torch.full((B, cols * (P if raw else 1)), -1, dtype=torch.int32)
        self.slots, at = [], 0
        for b, L in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            sl = [mine[t // P] * P + t % P for t in range(L)]
            self.slots.append(sl)
            rows = torch.randn((L, self.W), generator=g) * mag
            self.buf[layer].view(-1, self.W)[torch.tensor(sl, dtype=torch.long)] = rows.to(self.dt)
            if raw:
                table[b, :len(mine) * P] = torch.tensor([p * P + o for p in mine for o in range(P)])
            else:
                table[b, :len(mine)] = torch.tensor(mine)
        self.layer = layer
        self.buf, self.table = self.buf.to(DEV), table.to(DEV)
        self.pool = kb.LatentPool(self.buf, dc, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32)
        self.q = torch.randn((B, C, H, self.W), generator=g).to(self.dt).to(DEV)
        self.out = torch.full((B, C, H, dc), 5.0, dtype=self.dt, device=DEV)
        self.scale = 1.0 / math.sqrt(self.W)
        self.ws = kb.alloc_latent_workspace(self.pool, B, C, H, device=DEV)
        self.ws.fill_(0xFF)  # NaN as floats: its contents must not matter
        self.clens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def run(self, window=0, sinks=0, q_lens=None, **kw):
        self.kb.paged_latent_attention(self.pool, self.layer, self.q, self.table,
                                       self.kb.KVP_RAW_LOCATIONS if self.raw else self.kb.KVP_BLOCK_TABLE, self.clens,
                                       window, self.scale, self.out, self.ws, sinks=sinks,
                                       q_lens=None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device=DEV),
                                       **kw)
        torch.cuda.synchronize()
        return self.out

    def want(self, b, j, ql, window=0, sinks=0):
        p = self.lens[b] - ql + j
        sl = torch.tensor([self.slots[b][t] for t in R.span(p, window, sinks)], device=DEV)
        x = self.buf[self.layer].view(-1, self.W)[sl].double().cpu()
        return R.attend(self.q[b, j].double().cpu(), x, x[:, :self.dc], self.scale, self.dt)

    def verify(self, window=0, sinks=0, q_lens=None, only=None):
        out = self.out.cpu()
        for b in range(len(self.lens)) if only is None else only:
            ql = self.C if q_lens is None else q_lens[b]
            js = range(ql) if ql <= 12 else sorted({0, 1, ql // 3, ql // 2, ql - 2, ql - 1})
            for j in js:
                w, bound = self.want(b, j, ql, window, sinks)
                R.check(out[b, j], w, bound, f"request {b} query {j}")
            assert bool((out[b, ql:] == 5.0).all()), f"request {b}: rows past its queries were written"


CASES = [
    # dtype, lens, C, H, dc, dr, P, raw, window, sinks
    ("bf16", [1], 1, 16, 512, 64, 16, False, 0, 0),
    ("bf16", [777], 1, 16, 512, 64, 16, False, 0, 0),
    ("bf16", [1, 7, 8, 9, 63, 64, 65, 127, 128, 129, 200], 1, 16, 512, 64, 16, False, 0, 0),
    ("bf16", [1, 2, 63, 64, 65, 1000], 1, 64, 512, 64, 16, False, 0, 0),
    ("bf16", [5, 300, 4097], 1, 32, 512, 64, 64, False, 0, 0),
    ("bf16", [64, 900, 33], 1, 128, 512, 64, 16, False, 0, 0),      # two row tiles of a token
    ("bf16", [500, 130], 1, 40, 512, 64, 16, False, 0, 0),          # a tile with idle rows
    ("bf16", [500, 130], 1, 1, 512, 64, 16, False, 0, 0),
    ("bf16", [500, 130], 1, 3, 512, 64, 16, False, 0, 0),
    ("bf16", [500, 130, 71], 1, 16, 512, 64, 1, True, 0, 0),        # scattered rows
    ("bf16", [500, 130, 71], 1, 16, 512, 64, 1, False, 0, 0),
    ("bf16", [500, 130, 71], 1, 16, 512, 64, 4, False, 0, 0),       # pages smaller than a group
    ("bf16", [500, 130, 71], 1, 16, 512, 64, 12, False, 0, 0),      # and not a multiple of it
    ("bf16", [500, 130, 71], 1, 16, 512, 64, 24, True, 0, 0),
    ("bf16", [500, 130, 71], 1, 48, 512, 64, 8, False, 0, 0),
    ("bf16", [4, 66, 700], 4, 64, 512, 64, 16, False, 0, 0),        # verify
    ("bf16", [7, 70, 350], 7, 8, 512, 64, 16, False, 0, 0),
    ("bf16", [5, 64, 69], 5, 40, 512, 64, 16, False, 0, 0),         # tiles that cut a token's heads
    ("bf16", [300, 411], 130, 16, 512, 64, 16, False, 0, 0),        # a chunk: many tiles a request
    ("bf16", [260], 100, 128, 512, 64, 16, False, 0, 0),
    ("bf16", [3, 64, 100, 1000], 1, 16, 512, 64, 16, False, 50, 0),  # window
    ("bf16", [3, 64, 100, 1000], 1, 16, 512, 64, 16, False, 50, 2),  # and sinks
    ("bf16", [3, 64, 100, 1000], 3, 32, 512, 64, 16, False, 70, 17),
    ("bf16", [300, 411], 130, 16, 512, 64, 4, True, 33, 5),
    ("bf16", [5, 90], 1, 4, 128, 32, 4, False, 0, 0),               # other dims: the general kernel
    ("bf16", [5, 90], 2, 4, 100, 12, 4, True, 20, 3),
    ("bf16", [5, 90], 1, 2, 1024, 0, 4, False, 0, 0),
    ("f32", [1, 33, 300], 1, 16, 512, 64, 16, False, 0, 0),
    ("f32", [2, 40, 77], 2, 4, 64, 16, 4, True, 0, 0),
    ("f32", [2, 40, 77], 2, 4, 64, 16, 4, False, 9, 2),
]


@pytest.mark.parametrize("dtype,lens,C,H,dc,dr,P,raw,window,sinks", CASES)
def test_latent_attention_is_the_formula(kb, dtype, lens, C, H, dc, dr, P, raw, window, sinks):
    c = Case(kb, dtype, lens, C, H, dc, dr, P, raw, seed=C + H)
    c.run(window, sinks)
    c.verify(window, sinks)
    assert kb.kvp_sync_error(c.pool) == 0


def test_one_long_request_is_split(kb):
    """One request over every SM: partials and their join, twice, on a workspace of NaN."""
    c = Case(kb, "bf16", [30011], 1, 16, 512, 64, 16, seed=3)
    c.run()
    first = c.out.clone()
    c.verify()
    c.run()
    assert torch.equal(first, c.out), "the same call gives the same bits"


def test_more_requests_than_threads(kb):
    lens = [1 + (37 * i) % 90 for i in range(1500)]
    c = Case(kb, "bf16", lens, 1, 8, 512, 64, 16, seed=5)
    c.run()
    c.verify(only=list(range(0, 1500, 97)) + [1498, 1499])


def test_ragged_chunks_and_table_rows(kb):
    c = Case(kb, "bf16", [40, 300, 129, 64], 20, 16, 512, 64, 16, seed=6)
    ql = [20, 1, 13, 7]
    c.run(q_lens=ql)
    c.verify(q_lens=ql)
    perm = [2, 0, 3, 1]
    rows = torch.tensor(perm, dtype=torch.int32, device=DEV)
    table = torch.full_like(c.table, -1)
    for b, r in enumerate(perm):
        table[r] = c.table[b]
    keep, c.table = c.out.clone(), table
    c.out.fill_(5.0)
    c.run(q_lens=ql, table_rows=rows)
    assert torch.equal(keep, c.out)


def test_large_scores_and_late_maximum(kb):
    """Scores of hundreds, the largest at the end of the context: the running maximum grows block after block."""
    c = Case(kb, "bf16", [700, 90], 2, 16, 512, 64, 16, seed=7)
    flat = c.buf[0].view(-1, c.W)
    for b, L in enumerate(c.lens):
        sl = torch.tensor(c.slots[b], device=DEV)
        ramp = torch.linspace(0.01, 6.0, L, device=DEV)[:, None]
        flat[sl] = (c.q[b, 0, 0].float()[None] * ramp + 0.01 * flat[sl].float()).to(c.dt)
    c.run()
    c.verify()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window,sinks,at", [(0, 0, -3), (64, 0, -68), (64, 3, -68), (64, 3, -65), (64, 0, -2)])
@pytest.mark.parametrize("dtype,C,H,dc,dr,part", [("bf16", 5, 40, 512, 64, 7), ("bf16", 5, 8, 512, 64, 575),
                                                  ("bf16", 20, 64, 512, 64, 511), ("f32", 5, 4, 64, 16, 3)])
def test_a_row_that_is_not_finite_reaches_only_who_attends_it(kb, bad, window, sinks, at, dtype, C, H, dc, dr, part):
    """One entry of a row that some queries attend and others do not (later, or out of the window)."""
    c = Case(kb, dtype, [300, 90, 129], C, H, dc, dr, 16, seed=13)
    for b, L in enumerate(c.lens):
        c.buf[0].view(-1, c.W)[c.slots[b][L + at], part] = bad
    c.run(window, sinks)
    assert kb.kvp_sync_error(c.pool) == 0
    seen = [0, 0]
    for b, L in enumerate(c.lens):
        for j in range(C):
            attends = L + at in R.span(L - C + j, window, sinks)
            seen[attends] += 1
            if attends:
                assert not math.isnan(bad) or bool(c.out[b, j].isnan().all())
            else:
                R.check(c.out[b, j], *c.want(b, j, C, window, sinks), f"request {b} query {j}")
    assert seen[0] and (seen[1] or at == -68)  # with 3 sinks and 5 queries that row has left all windows


def test_a_query_that_is_not_finite_stays_alone(kb):
    for bad in (float("nan"), float("inf")):
        c = Case(kb, "bf16", [300, 90, 6], 5, 40, 512, 64, 16, seed=14)
        c.q[0, 2, 7, 5] = c.q[1, 4, 39, 575] = c.q[2, 0, 0, 0] = bad
        c.run()
        out = c.out.cpu()
        for b in range(3):
            for j in range(5):
                w, bound = c.want(b, j, 5)
                ok = w.isfinite().all(-1)
                R.check(out[b, j][ok], w[ok], bound[ok], f"request {b} query {j}")
                assert int(ok.sum()) == 40 - (j == (2, 4, 0)[b])


@pytest.mark.parametrize("P", [16, 1])
def test_rows_past_four_gigabytes(kb, P):
    """Stored by rotary_store_latent and attended at offsets that 32 bits do not hold, in the second layer."""
    dc, dr, H, slots = 512, 64, 16, 2_000_000
    W, g = dc + dr, torch.Generator().manual_seed(P)
    buf = torch.empty((2, slots // P, P, W), dtype=torch.bfloat16, device=DEV)
    assert 2 * slots * W > 2 ** 31
    pool = kb.LatentPool(buf, dc, kb.KVP_BF16)
    L = 150
    pages = slots // P - 1 - torch.randperm(-(-L // P) + 5, generator=g)[:-(-L // P)]
    sl = torch.tensor([int(pages[t // P]) * P + t % P for t in range(L)], dtype=torch.int32, device=DEV)
    rows = torch.randn((L, W), generator=g).bfloat16().to(DEV)
    kb.rotary_store_latent(pool, 1, None, rows[:, :dc], rows[:, dc:], torch.zeros(L, dtype=torch.int32, device=DEV), sl,
                           kb.RotaryPlan(dr, device=DEV), None)
    assert torch.equal(buf[1].view(slots, W)[sl.long()], rows)  # position 0 turns nothing
    q = torch.randn((1, 1, H, W), generator=g).bfloat16().to(DEV)
    out = torch.empty((1, 1, H, dc), dtype=torch.bfloat16, device=DEV)
    kb.paged_latent_attention(pool, 1, q, pages.to(torch.int32)[None].to(DEV), kb.KVP_BLOCK_TABLE,
                              torch.tensor([L], dtype=torch.int32, device=DEV), 0, W ** -0.5, out,
                              kb.alloc_latent_workspace(pool, 1, 1, H, device=DEV))
    x = rows.double().cpu()
    R.check(out[0, 0], *R.attend(q[0, 0].double().cpu(), x, x[:, :dc], W ** -0.5, torch.bfloat16))
    assert kb.kvp_sync_error(pool) == 0


def test_the_widest_windows(kb):
    """Windows at and past what the table can hold, to the end of int32."""
    for dc, dr, H in ((512, 64, 40), (64, 16, 3)):
        c = Case(kb, "bf16", [300, 90, 7], 5, H, dc, dr, 16, seed=15)
        full = c.run().clone()
        cap = c.table.shape[1] * 16
        for window, sinks in ((cap, 0), (cap + 1, 3), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 2)):
            c.out.fill_(5.0)
            assert torch.equal(c.run(window, sinks), full)
        c.run(cap - 1, 0)
        c.verify(cap - 1, 0)


def test_bad_requests_and_pages(kb):
    """An invalid length or table row zero-fills its request, a hole is skipped, and the others are untouched by it."""
    for dc, dr, H in ((512, 64, 16), (128, 32, 4)):
        lens = [100, 50, 300, 64]
        c = Case(kb, "bf16", lens, 1, H, dc, dr, 16, seed=9)
        c.clens[1] = 0
        c.run()
        assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
        c.verify(only=[0, 2, 3])
        assert bool((c.out[1] == 0).all())
        c.clens[1] = c.table.shape[1] * 16 + 1
        c.run()
        assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
        c.verify(only=[0, 2, 3])
        assert bool((c.out[1] == 0).all())
        c.clens[1] = 50
        c.run(table_rows=torch.tensor([0, 4, 2, -1], dtype=torch.int32, device=DEV))
        assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
        c.verify(only=[0, 2])
        assert bool((c.out[1] == 0).all()) and bool((c.out[3] == 0).all())
        for bad in (-1, c.pool.num_pages, 2 ** 31 - 1):
            c.table[2, 3] = bad
            c.run()
            assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
            c.verify(only=[0, 1, 3])
        q_lens = [1, 2, 1, 1]
        c.table[2, 3] = c.table[2, 2]
        c.run(q_lens=q_lens)
        assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
        assert bool((c.out[1] == 0).all())


def test_layers_streams_and_graphs(kb):
    a = Case(kb, "bf16", [333, 64, 1200], 1, 32, 512, 64, 16, seed=11, layers=3, layer=1)
    b = Case(kb, "bf16", [900, 10], 2, 64, 512, 64, 4, raw=True, seed=12)
    a.run(), b.run()
    a.verify(), b.verify()
    wa, wb = a.out.clone(), b.out.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for o in (a.out, b.out):
        o.fill_(5.0)
    torch.cuda.synchronize()
    call = lambda c, s=None: kb.paged_latent_attention(c.pool, c.layer, c.q, c.table,  # noqa: E731
                                                       kb.KVP_RAW_LOCATIONS if c.raw else kb.KVP_BLOCK_TABLE, c.clens, 0,
                                                       c.scale, c.out, c.ws, stream=s)
    for _ in range(5):  # two calls at once, each with its own workspace
        call(a, s1)
        call(b, s2)
    torch.cuda.synchronize()
    assert torch.equal(a.out, wa) and torch.equal(b.out, wb)
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(c)
            call(c)
        graphs.append(g)
    for o in (a.out, b.out):
        o.fill_(5.0)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, wa) and torch.equal(b.out, wb)
    a.clens -= 7  # a replay follows the lengths
    a.lens = [x - 7 for x in a.lens]
    graphs[0].replay()
    torch.cuda.synchronize()
    a.verify()


def test_refusals(kb):
    c = Case(kb, "bf16", [100], 1, 16, 512, 64, 16, seed=1)
    call = lambda q=c.q, out=c.out, ws=c.ws, lens=c.clens, scale=1.0, window=0, sinks=0, layer=0, mode=0, pool=c.pool: (  # noqa: E731
        kb.paged_latent_attention(pool, layer, q, c.table, mode, lens, window, scale, out, ws, sinks=sinks))
    for kw in (dict(q=c.q.float()), dict(out=c.out.float()), dict(lens=c.clens.long())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=c.q[..., :512]), dict(out=c.q), dict(lens=torch.cat((c.clens, c.clens)))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(ws=None), dict(ws=c.ws[:128]), dict(ws=c.ws[1:]), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(window=4, sinks=4), dict(sinks=-1), dict(layer=1), dict(layer=-1), dict(mode=2)):
        with pytest.raises(kb.KvpError) as e:
            call(**kw)
        assert e.value.code == kb.KVP_ERR_INVALID_ARG
    kv = kb.Pool(torch.zeros((2, 1, 4, 16, 1, 576), dtype=torch.bfloat16, device=DEV), 16, kb.KVP_BF16)
    with pytest.raises(AttributeError):
        call(pool=kv)  # a K/V pool has no latent_dim
    torch.cuda.synchronize()
    assert bool((c.out == 5.0).all()) and kb.kvp_sync_error(c.pool) == 0


def test_negative_and_zero_scale(kb):
    for scale in (-0.05, 0.0):
        c = Case(kb, "bf16", [100, 37], 1, 16, 512, 64, 16, seed=2)
        c.scale = scale
        c.run()
        c.verify()


@pytest.mark.parametrize("C,H,L", [(1, 16, 3000), (1, 32, 1500), (4, 64, 900), (20, 64, 640)])
def test_a_maximum_that_grows_in_some_rows_of_every_block(kb, C, H, L):
    """O is scaled in each block, for other rows each time, so that the warps that scale it and those that do not are
    never in step: the formula, and the same bits every time."""
    c = Case(kb, "bf16", [L, L // 2], C, H, 512, 64, 16, seed=16)
    flat = c.buf[0].view(-1, c.W)
    for b, n in enumerate(c.lens):
        sl = torch.tensor(c.slots[b], device=DEV)
        # block i grows with the query of head i mod H, by 9 and more in log2 units of that head's scores
        which = (torch.arange(n, device=DEV) // 64) % H
        size = (1 + torch.arange(n, device=DEV) // 64)[:, None] * 8.0 / (c.scale * c.W)
        flat[sl] = (c.q[b, 0, which].float() * size + 0.1 * flat[sl].float()).to(c.dt)
    c.run()
    c.verify()
    first = c.out.clone()
    for _ in range(30):
        c.out.fill_(5.0)
        c.run()
        assert torch.equal(c.out, first)
    assert kb.kvp_sync_error(c.pool) == 0


NOT_FINITE = [
    # dtype, lens, C, H, dc, dr, P, window, sinks, position of the row from the end
    ("bf16", [300, 90, 131], 1, 64, 512, 64, 16, 0, 0, -1),     # in the last block of 64 keys
    ("bf16", [300, 90, 131], 1, 64, 512, 64, 16, 0, 0, -80),    # in a block that every query attends
    ("bf16", [300, 91, 131], 1, 16, 512, 64, 1, 0, 0, -80),
    ("bf16", [300, 90, 131], 5, 40, 512, 64, 16, 0, 0, -80),
    ("bf16", [300, 90, 131], 5, 40, 512, 64, 16, 0, 0, -3),     # newer than some queries
    ("bf16", [300, 90, 131], 20, 64, 512, 64, 16, 0, 0, -12),
    ("bf16", [300, 90, 131], 3, 32, 512, 64, 16, 70, 2, -70),   # at the window's edge
    ("bf16", [5000], 1, 16, 512, 64, 16, 0, 0, -2000),          # a split request
    ("bf16", [5000], 4, 16, 512, 64, 16, 0, 0, -3),
    ("bf16", [70, 33], 3, 4, 128, 32, 4, 0, 0, -2),             # the general kernel
    ("f32", [70, 33], 3, 4, 64, 16, 4, 0, 0, -20),
    ("f32", [70, 33], 3, 4, 64, 16, 4, 9, 2, -10),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("dtype,lens,C,H,dc,dr,P,window,sinks,at", NOT_FINITE)
def test_who_attends_a_row_that_is_not_finite_is_nan(kb, bad, rope, dtype, lens, C, H, dc, dr, P, window, sinks, at):
    """Wherever the row lies and whatever its score: heads that meet an infinity with the other sign score minus
    infinity, a weight of zero, and are NaN all the same."""
    c = Case(kb, dtype, lens, C, H, dc, dr, P, seed=21)
    part = dc + 3 if rope else dc // 2 + 1
    for b, L in enumerate(lens):
        c.buf[0].view(-1, c.W)[c.slots[b][L + at], part] = bad
    c.run(window, sinks)
    assert kb.kvp_sync_error(c.pool) == 0
    for b, L in enumerate(lens):
        for j in range(C):
            if L + at in R.span(L - C + j, window, sinks):
                assert bool(c.out[b, j].isnan().all()), f"request {b} query {j}"
            else:
                R.check(c.out[b, j], *c.want(b, j, C, window, sinks), f"request {b} query {j}")


@pytest.mark.parametrize("dtype,C,H,dc,dr", [("bf16", 1, 16, 512, 64), ("bf16", 5, 40, 512, 64), ("f32", 2, 4, 64, 16)])
def test_a_score_past_fp32_of_a_finite_row_weighs_nothing(kb, dtype, C, H, dc, dr):
    """A finite row whose score overflows to minus infinity counts as the formula has it: not at all."""
    c = Case(kb, dtype, [200, 67], C, H, dc, dr, 16, seed=22)
    c.q[..., 3] = -100.0
    rows = c.buf[0].view(-1, c.W)
    for b, L in enumerate(c.lens):
        rows[torch.tensor(c.slots[b], device=DEV), 3] = 0
        for t in (5, L - C):  # one that all rows' blocks attend, one in the last block
            rows[c.slots[b][t], 3] = 3e38
    c.run()
    for b, L in enumerate(c.lens):
        for j in range(C):
            sl = torch.tensor([c.slots[b][t] for t in range(L - C + j + 1) if t not in (5, L - C)], device=DEV)
            x = rows[sl].double().cpu()
            w, bound = R.attend(c.q[b, j].double().cpu(), x, x[:, :dc], c.scale, c.dt)
            R.check(c.out[b, j], w, bound, f"request {b} query {j}")


def test_the_cache_has_one_workspace_for_all_shapes(kb):
    """Many batches and chunk lengths take no more memory than the largest few, and a graph captured on a smaller
    workspace replays after larger calls have come."""
    from paged_decode_attention_store_gb300.engine import PagedLatentCache

    dc, dr, H = 512, 64, 8
    cache = PagedLatentCache(64, 16, dc, dr, 1, max_requests=8)
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)  # noqa: E731
    rope = kb.RotaryPlan(dr, device=DEV)
    cache.new(0)
    L = 200
    slots = cache.append([0] * L)
    cache.store(0, None, rnd(L, dc), rnd(L, dr), torch.arange(L, dtype=torch.int32, device=DEV), slots, rope, None)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    scale = (dc + dr) ** -0.5
    x = cache.rows(0, [0])[0].double().cpu()

    def right(q, out):
        C = q.shape[1]
        for j in {0, C - 1}:
            keys = x[:L - C + j + 1]
            R.check(out[0, j], *R.attend(q[0, j].double().cpu(), keys, keys[:, :dc], scale, torch.bfloat16))

    q1, out1 = rnd(1, 1, H, dc + dr), torch.empty((1, 1, H, dc), dtype=torch.bfloat16, device=DEV)
    cache.attend(0, q1, lens, 0, scale, out1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(0, q1, lens, 0, scale, out1)
    held = torch.cuda.memory_allocated()
    sizes = set()
    for B in range(1, 33):
        for C in (1, 2, 3, 5, 8, 33, 64):
            need = kb.paged_latent_attention_workspace_size(cache.pool, B, C, H)
            assert cache.workspace(B, H, C).nbytes >= need
            sizes.add(need)
    assert len({t.data_ptr() for t in cache._ws.values()}) <= len(sizes) <= 6
    assert torch.cuda.memory_allocated() - held <= sum(sizes) + 512 * len(sizes)
    for C in (1, 3, 64, 150, 2):
        q, out = rnd(1, C, H, dc + dr), torch.empty((1, C, H, dc), dtype=torch.bfloat16, device=DEV)
        cache.attend(0, q, lens, 0, scale, out)
        right(q, out)
    out1.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    right(q1, out1)
    cache.check()
