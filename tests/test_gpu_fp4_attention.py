"""paged_fp4_attention against the 64-bit formulas."""

import math

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from libbuild import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FEW = 64  # (token, head) columns a KV head up to which a call is the decode kernel's, with fp16 weights


@pytest.fixture(scope="module")
def kb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_built()


class Case:
    """Requests of the given lengths on shuffled pages; every slot that holds no token reads as NaN."""

    def __init__(self, kb, dtype, lens, C, H, hkv, D, P, raw=False, seed=0, layers=1, layer=0, spare=3, gk=1.0, gv=1.0,
                 shuffle_slots=False, mag=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kb, self.dt, self.lens, self.C, self.H, self.hkv, self.D, self.raw = kb, DT[dtype], list(lens), C, H, hkv, D, raw
        need = [-(-max(L, 1) // P) for L in lens]
        pages = sum(need) + spare
        self.pool = kb.kv_fp4_pool_create(pages, P, hkv, D, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32, layers, gk, gv,
                                          device=DEV)
        self.pool.codes.fill_(0x77)
        self.pool.scales.fill_(0x7F)
        order = torch.randperm(pages, generator=g).tolist()
        B, cols = len(lens), max(need) + 1
        table = torch.full((B, cols * (P if raw else 1)), -1, dtype=torch.int32)
        self.slots, at = [], 0
        for b, L in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            sl = [p * P + o for p in mine for o in range(P)]
            if shuffle_slots:
                sl = [sl[i] for i in torch.randperm(len(sl), generator=g).tolist()]
            if raw:
                table[b, :len(sl)] = torch.tensor(sl)
            else:
                table[b, :len(mine)] = torch.tensor(mine)
            self.slots.append(sl[:L])
        self.layer, self.table = layer, table.to(DEV)
        flat = torch.tensor([s for sl in self.slots for s in sl], dtype=torch.int32)
        kv = (torch.randn((len(flat), 2 * hkv, D), generator=g) * mag).to(self.dt).to(DEV)
        if len(flat):
            kb.store_cache_fp4(self.pool, layer, kv[:, :hkv], kv[:, hkv:], flat.to(DEV))
        self.q = torch.randn((B, C, H, D), generator=g).to(self.dt).to(DEV)
        self.out = torch.full((B, C, H, D), 5.0, dtype=self.dt, device=DEV)
        self.scale = 1.0 / math.sqrt(D)
        self.most = max(max(lens), 1)
        self.ws = kb.alloc_fp4_workspace(self.pool, B, C, H, self.most, device=DEV)
        self.ws.fill_(0xFF)  # NaN as floats: its contents must not matter
        self.clens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.gk, self.gv = gk, gv
        self.read()

    def read(self):
        codes, scales = F.unpack(self.pool, self.layer)
        self.k = F.values(codes[:, :, 0], scales[:, :, 0], self.gk)
        self.v = F.values(codes[:, :, 1], scales[:, :, 1], self.gv)

    def run(self, window=0, sinks=0, q_lens=None, **kw):
        self.kb.paged_fp4_attention(self.pool, self.layer, self.q, self.table,
                                    self.kb.KVP_RAW_LOCATIONS if self.raw else self.kb.KVP_BLOCK_TABLE, self.clens, window,
                                    self.scale, self.out, self.ws, sinks=sinks, max_context=self.most,
                                    q_lens=None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device=DEV), **kw)
        torch.cuda.synchronize()
        return self.out

    def want(self, b, j, ql, window=0, sinks=0):
        sl = torch.tensor([self.slots[b][t] for t in R.span(self.lens[b] - ql + j, window, sinks)])
        G = self.H // self.hkv
        each = [F.attend(self.q[b, j, h * G:(h + 1) * G].double().cpu(), self.k[sl, h], self.v[sl, h], self.scale, self.dt,
                         torch.float16 if self.C * G <= FEW else torch.bfloat16)
                for h in range(self.hkv)]
        return torch.cat([x[0] for x in each]), torch.cat([x[1] for x in each])

    def verify(self, window=0, sinks=0, q_lens=None, only=None, few=False):
        out = self.out.cpu()
        for b in range(len(self.lens)) if only is None else only:
            ql = self.C if q_lens is None else q_lens[b]
            js = range(ql) if ql <= 12 and not few else sorted({0, ql // 3, ql // 2, max(0, ql - 2), ql - 1})
            for j in js:
                w, bound = self.want(b, j, ql, window, sinks)
                R.check(out[b, j], w, bound, f"request {b} query {j}")
            assert bool((out[b, ql:] == 5.0).all()), f"request {b}: rows past its queries were written"


CASES = [
    # dtype, lens, C, H, hkv, D, P, raw, window, sinks
    ("bf16", [1], 1, 32, 8, 128, 16, False, 0, 0),
    ("bf16", [777], 1, 32, 8, 128, 16, False, 0, 0),
    ("bf16", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200], 1, 32, 8, 128, 16, False, 0, 0),
    ("bf16", [1, 31, 64, 1000], 1, 8, 8, 128, 16, False, 0, 0),
    ("bf16", [1, 31, 64, 1000], 1, 64, 8, 128, 16, False, 0, 0),
    ("bf16", [1, 31, 64, 1000], 1, 128, 8, 128, 16, False, 0, 0),   # sixteen columns a head
    ("bf16", [33, 500], 1, 80, 8, 128, 16, False, 0, 0),            # ten
    ("bf16", [33, 500], 1, 12, 4, 128, 16, False, 0, 0),            # three
    ("bf16", [33, 500], 1, 8, 2, 128, 16, False, 0, 0),
    ("bf16", [33, 500], 1, 8, 1, 128, 16, False, 0, 0),
    ("bf16", [33, 500], 1, 71, 1, 128, 16, False, 0, 0),
    ("bf16", [33, 500], 1, 5, 5, 128, 16, False, 0, 0),             # five heads
    ("bf16", [33, 500], 1, 32, 16, 128, 16, False, 0, 0),           # two groups of eight heads
    ("bf16", [33, 500], 1, 24, 12, 128, 16, False, 0, 0),           # two of six
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 1, True, 0, 0),          # scattered rows
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 1, False, 0, 0),
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 4, False, 0, 0),         # pages smaller than a group
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 24, False, 0, 0),        # not a multiple of it
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 24, True, 0, 0),
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 32, True, 0, 0),
    ("bf16", [33, 500, 71], 1, 32, 8, 128, 64, False, 0, 0),
    ("bf16", [33, 500, 71], 1, 16, 16, 128, 3, True, 0, 0),
    ("bf16", [4, 66, 700], 4, 32, 8, 128, 16, False, 0, 0),         # verify
    ("bf16", [7, 70, 350], 7, 8, 1, 128, 16, False, 0, 0),
    ("bf16", [5, 64, 69], 5, 40, 8, 128, 16, False, 0, 0),
    ("bf16", [12, 64, 169], 12, 64, 8, 128, 16, False, 0, 0),
    ("bf16", [32, 100], 32, 8, 8, 128, 4, True, 0, 0),
    ("bf16", [300, 411], 130, 32, 8, 128, 16, False, 0, 0),         # chunks
    ("bf16", [260], 100, 16, 1, 128, 16, False, 0, 0),
    ("bf16", [260, 129], 65, 24, 8, 128, 16, False, 0, 0),          # three columns a head: not the tiles of the chunk kernel
    ("bf16", [3, 64, 100, 1000], 1, 32, 8, 128, 16, False, 50, 0),  # window
    ("bf16", [3, 64, 100, 1000], 1, 32, 8, 128, 16, False, 50, 2),  # and sinks
    ("bf16", [40, 64, 100, 1000], 1, 32, 8, 128, 16, False, 70, 40),
    ("bf16", [3, 64, 100, 1000], 3, 32, 8, 128, 16, False, 70, 17),
    ("bf16", [300, 411], 130, 16, 4, 128, 4, True, 33, 5),
    ("bf16", [300, 411], 130, 16, 4, 128, 16, False, 64, 0),
    ("bf16", [5, 90], 1, 4, 2, 64, 4, False, 0, 0),                 # other widths: the general kernel
    ("bf16", [5, 90], 2, 8, 8, 16, 4, True, 20, 3),
    ("bf16", [5, 290], 1, 8, 2, 256, 16, False, 0, 0),
    ("f32", [1, 33, 300], 1, 16, 8, 128, 16, False, 0, 0),
    ("f32", [2, 40, 77], 2, 4, 4, 64, 4, True, 9, 2),
    ("f32", [60, 140], 50, 4, 1, 128, 16, False, 0, 0),
]


@pytest.mark.parametrize("dtype,lens,C,H,hkv,D,P,raw,window,sinks", CASES)
def test_attention_is_the_formula(kb, dtype, lens, C, H, hkv, D, P, raw, window, sinks):
    c = Case(kb, dtype, lens, C, H, hkv, D, P, raw, seed=C + H, gk=0.5, gv=2.0)
    c.run(window, sinks)
    c.verify(window, sinks)
    assert kb.kvp_sync_error(c.pool) == 0


@pytest.mark.parametrize("C,q_lens,lens", [(6, [1, 6, 3, 2], [5, 6, 64, 300]), (200, [200, 1, 77, 130], [200, 300, 77, 431])])
def test_ragged_queries(kb, C, q_lens, lens):
    for window, sinks in ((0, 0), (40, 3)):
        c = Case(kb, "bf16", lens, C, 32, 8, 128, 16, seed=4)
        c.run(window, sinks, q_lens=q_lens)
        c.verify(window, sinks, q_lens=q_lens)


def test_one_long_request_is_split(kb):
    """One request over every SM: partials and their join, twice, on a workspace of NaN; the same bits."""
    c = Case(kb, "bf16", [30011], 1, 32, 8, 128, 16, seed=3)
    first = c.run().clone()
    c.verify()
    c.ws.fill_(0x3C)
    c.run()
    assert torch.equal(first, c.out)


def test_locations_in_any_order(kb):
    """A raw table whose slots are shuffled within and across pages."""
    c = Case(kb, "bf16", [700, 65, 1], 1, 32, 8, 128, 32, raw=True, shuffle_slots=True, seed=8)
    c.run()
    c.verify()


def test_many_requests(kb):
    lens = [1 + (37 * i) % 90 for i in range(1500)]
    c = Case(kb, "bf16", lens, 1, 8, 8, 128, 16, seed=5)
    c.run()
    c.verify(only=[0, 1, 700, 1499])


def test_more_requests_than_a_block_plans(kb):
    """Tens of thousands of requests of a few tokens."""
    c = Case(kb, "bf16", [1 + i % 3 for i in range(20011)], 1, 2, 1, 128, 4, seed=5)
    c.run()
    c.verify(only=[0, 1, 2, 10000, 20010])


@pytest.mark.parametrize("C,H,hkv", [(1, 32, 8), (4, 32, 8), (140, 32, 8), (2, 4, 1)])
def test_bad_requests_are_zeros_and_recorded(kb, C, H, hkv):
    lens = [200, 0, 220, 170, 250]
    c = Case(kb, "bf16", [200, 1, 220, 170, 250], C, H, hkv, 128, 16, seed=6)
    c.clens.copy_(torch.tensor([200, 0, 100000, 170, 250]))
    rows = torch.tensor([0, 1, 2, 77, 4], dtype=torch.int32, device=DEV)
    c.run(table_rows=rows)
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    assert bool((c.out[1:4] == 0).all())
    c.verify(only=[0, 4])
    assert lens[0] == c.lens[0]


@pytest.mark.parametrize("C", [1, 4, 140])
def test_holes_are_skipped_and_recorded(kb, C):
    c = Case(kb, "bf16", [200, 220], C, 32, 8, 128, 16, seed=6)
    c.table[0, 3] = -1
    c.table[0, 5] = 1 << 30
    c.run()
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    c.verify(only=[1])


@pytest.mark.parametrize("C,H,hkv", [(1, 32, 8), (4, 32, 8), (7, 8, 1), (140, 32, 8), (30, 5, 5)])
def test_blocks_of_nan_reach_who_attends_them(kb, C, H, hkv):
    """NaN scales in K and V of the newest tokens: earlier queries of the same call do not see them."""
    lens = [180, 333]
    c = Case(kb, "bf16", lens, C, H, hkv, 128, 16, seed=7)
    cut = max(1, C // 2)  # the last ``cut`` - 1 tokens ...
    kt, vt = c.lens[0] - cut, c.lens[1] - cut
    for slot, head, part, block in ((c.slots[0][kt], 0, 0, 2), (c.slots[1][vt], hkv - 1, 1, 5)):
        c.pool.scales[0, slot // 16, head, slot % 16, part, block] = 0x7F
    c.run()
    G, out = H // hkv, c.out.float().cpu()
    for j in range(C):
        sees = j >= C - cut
        assert bool(out[0, j, :G].isnan().all()) == sees and bool(out[0, j, :G].isnan().any()) == sees, j
        assert not bool(out[0, j, G:].isnan().any())
        last = out[1, j, H - G:]
        assert bool(last[:, 80:96].isnan().all()) == sees and bool(last[:, 80:96].isnan().any()) == sees, j
        assert not bool(last[:, :80].isnan().any()) and not bool(last[:, 96:].isnan().any())
        assert not bool(out[1, j, :H - G].isnan().any())
    for b in range(2):
        for j in (0, C - cut - 1):
            if 0 <= j < C - cut:
                w, bound = c.want(b, j, C)
                R.check(c.out[b, j].cpu(), w, bound, f"request {b} query {j}")


@pytest.mark.parametrize("C", [1, 4])
def test_queries_of_any_size(kb, C):
    """Rows from 2^-100 to 2^100, zeros, and rows whose entries differ by far."""
    c = Case(kb, "bf16", [150, 99], C, 32, 8, 128, 16, seed=9)
    for h, e in ((0, -100), (1, -40), (2, 20), (3, 100)):
        c.q[:, :, h] *= 2.0 ** e
    c.q[:, :, 4] = 0
    c.q[:, :, 5, ::3] *= 2.0 ** -30
    c.run()
    out = c.out.cpu()
    assert not bool(out.isnan().any())
    for b in range(2):
        for j in range(C):
            w, bound = c.want(b, j, C)
            keep = [h for h in range(32) if h not in (2, 3)]
            R.check(out[b, j, keep], w[keep], bound[keep])
            # one key has all the weight: its value, rounded once
            R.check(out[b, j, 3], w[3], R.u(torch.bfloat16) * w[3].abs() + 1e-30)


def test_queries_that_are_not_finite(kb):
    c = Case(kb, "bf16", [150], 1, 32, 8, 128, 16, seed=9)
    c.q[0, 0, 3, 7] = float("nan")
    c.q[0, 0, 9, 7] = float("inf")
    c.run()
    bad = c.out[0, 0].isnan().all(-1)
    assert bool(bad[3]) and bool(bad[9])
    keep = [h for h in range(32) if h not in (3, 9)]
    w, bound = c.want(0, 0, 1)
    R.check(c.out[0, 0, keep].cpu(), w[keep], bound[keep])


def test_scores_that_climb(kb):
    """Scores that rise along the context: the running maximum is raised again and again; scales of either sign."""
    c = Case(kb, "bf16", [2000, 700], 1, 32, 8, 128, 16, seed=10, mag=3.0)
    c.q *= 4
    for scale in (c.scale, -c.scale, 0.0):
        c.scale = scale
        c.run()
        c.verify()


@pytest.mark.parametrize("C", [1, 4, 140])
def test_captured_and_replayed(kb, C):
    c = Case(kb, "bf16", [300, 411], C, 32, 8, 128, 16, seed=12)
    want = c.run().clone()
    lens = c.clens.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    rows = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    with torch.cuda.graph(g, stream=s):
        kb.paged_fp4_attention(c.pool, 0, c.q, c.table, kb.KVP_BLOCK_TABLE, c.clens, 0, c.scale, c.out, c.ws,
                               max_context=c.most, table_rows=rows)
    c.out.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)
    c.clens.copy_(torch.tensor([200, 141]))
    g.replay()
    torch.cuda.synchronize()
    c.lens = [200, 141]
    c.verify()
    c.clens.copy_(lens)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_another_stream(kb):
    c = Case(kb, "bf16", [300, 411], 1, 32, 8, 128, 16, seed=12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    c.verify()


def test_rows_past_four_gigabytes(kb):
    """A pool whose bytes pass 32 bits, the context in its last pages, the second of two layers."""
    hkv, D, P = 8, 128, 16
    pages = (1 << 32) // (hkv * D * P) + 300
    pool = kb.kv_fp4_pool_create(pages, P, hkv, D, kb.KVP_BF16, 2, device=DEV)
    g = torch.Generator().manual_seed(10)
    L = 500
    table = (pages - 1 - torch.arange(-(-L // P))).to(torch.int32)[None]
    slots = (table[0].long()[:, None] * P + torch.arange(P)).flatten()[:L]
    x = torch.randn((L, 2 * hkv, D), generator=g).to(torch.bfloat16)
    d = x.to(DEV)
    kb.store_cache_fp4(pool, 1, d[:, :hkv], d[:, hkv:], slots.to(torch.int32).to(DEV))
    for C in (1, 140):
        q = torch.randn((1, C, 32, D), generator=g).to(torch.bfloat16).to(DEV)
        out = torch.zeros_like(q)
        ws = kb.alloc_fp4_workspace(pool, 1, C, 32, L, device=DEV)
        kb.paged_fp4_attention(pool, 1, q, table.to(DEV), kb.KVP_BLOCK_TABLE, torch.tensor([L], dtype=torch.int32, device=DEV),
                               0, D ** -0.5, out, ws, max_context=L)
        assert kb.kvp_sync_error(pool) == 0
        for h in (0, 31):
            k, v = (F.values(*F.quantise(x[:, p * hkv + h // 4].double(), 1.0), 1.0) for p in (0, 1))
            w, bound = F.attend(q[0, -1, h][None].double().cpu(), k, v, D ** -0.5, torch.bfloat16,
                                torch.float16 if C == 1 else torch.bfloat16)
            R.check(out[0, -1, h][None].cpu(), w, bound)
