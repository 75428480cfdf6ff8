"""latent_prefill_attention against the 64-bit formulas, and against the absorbed form."""

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
    def __init__(self, kb, dtype, ql, kl, H, dn, dr, dv, seed=0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.kb, self.dt, self.ql, self.kl, self.H, self.dn, self.dr, self.dv = kb, DT[dtype], ql, kl, H, dn, dr, dv
        tq, tk = sum(ql) + extra, sum(kl) + extra
        rnd = lambda *s: torch.randn(s, generator=g).to(self.dt).to(DEV)  # noqa: E731
        up = rnd(tk, H, dn + dv)
        self.k, self.v = up[..., :dn], up[..., dn:]
        self.pe = rnd(tk, 40 + dr)[:, 40:] if dr else None
        self.q = rnd(tq, H, dn + dr)
        if extra:  # rows that no request owns
            self.q[-extra:] = float("nan")
            up[-extra:] = float("nan")
            if dr:
                self.pe[-extra:] = float("nan")
        start = lambda xs: [sum(xs[:i]) for i in range(len(xs) + 1)]  # noqa: E731
        self.q0, self.k0 = start(ql), start(kl)
        self.qs = torch.tensor(self.q0, dtype=torch.int32, device=DEV)
        self.ks = torch.tensor(self.k0, dtype=torch.int32, device=DEV)
        self.out = torch.full((tq, H, dv), 5.0, dtype=self.dt, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.scale, self.max_q = 1.0 / math.sqrt(dn + dr), max(ql)

    def run(self, **kw):
        self.kb.latent_prefill_attention(self.q, self.k, self.pe, self.v, self.qs, self.ks, self.max_q, self.scale, self.out,
                                         error_word=self.err, **kw)
        torch.cuda.synchronize()

    def verify(self, only=None):
        out, q, v = self.out.cpu(), self.q.double().cpu(), self.v.double().cpu()
        key = self.k.double().cpu()
        if self.dr:
            key = torch.cat((key, self.pe.double().cpu()[:, None].expand(-1, self.H, -1)), -1)
        for b in range(len(self.ql)) if only is None else only:
            n, m = self.ql[b], self.kl[b]
            js = range(n) if n <= 16 else sorted({0, 1, 16, n // 2, n - 2, n - 1, min(127, n - 1), min(128, n - 1)})
            for j in js:
                keys = slice(self.k0[b], self.k0[b] + m - n + j + 1)
                w, bound = R.attend(q[self.q0[b] + j], key[keys], v[keys], self.scale, self.dt)
                R.check(out[self.q0[b] + j], w, bound, f"request {b} query {j}")
        assert bool((out[sum(self.ql):] == 5.0).all()), "rows behind the last request were written"


CASES = [
    # dtype, query rows, key rows, H, dn, dr, dv, extra rows
    ("bf16", [1], [1], 1, 128, 64, 128, 0),
    ("bf16", [1, 2, 5], [1, 2, 5], 4, 128, 64, 128, 3),
    ("bf16", [127, 128, 129], [127, 128, 129], 2, 128, 64, 128, 1),
    ("bf16", [33, 1, 600, 257], [33, 1, 600, 257], 16, 128, 64, 128, 0),
    ("bf16", [1, 1, 1], [1000, 128, 129], 8, 128, 64, 128, 0),       # single new tokens on long prefixes
    ("bf16", [64, 200, 3], [700, 200, 515], 5, 128, 64, 128, 200),
    ("bf16", [0, 40, 0, 7], [0, 40, 9, 300], 3, 128, 64, 128, 2),    # requests without queries, or without anything
    ("bf16", [300], [5000], 2, 128, 64, 128, 0),
    ("bf16", [40, 9], [40, 100], 3, 64, 32, 64, 1),                  # other dims: the general kernel
    ("bf16", [17], [30], 2, 192, 0, 100, 1),
    ("bf16", [5], [30], 2, 7, 5, 3, 1),
    ("f32", [33, 1, 100], [33, 50, 300], 4, 128, 64, 128, 2),
    ("f32", [20, 4], [20, 33], 2, 40, 8, 512, 0),
]


@pytest.mark.parametrize("dtype,ql,kl,H,dn,dr,dv,extra", CASES)
def test_expanded_attention_is_the_formula(kb, dtype, ql, kl, H, dn, dr, dv, extra):
    c = Case(kb, dtype, ql, kl, H, dn, dr, dv, seed=H, extra=extra)
    c.run()
    c.verify()
    assert int(c.err) == 0
    c.max_q += 1000  # an upper bound is fine
    first = c.out.clone()
    c.out.fill_(5.0)
    c.run()
    assert torch.equal(first, c.out) and int(c.err) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["v", "k", "pe", "q"])
@pytest.mark.parametrize("dtype,dn,dr,dv", [("bf16", 128, 64, 128), ("bf16", 64, 32, 64), ("f32", 128, 64, 128)])
def test_what_is_not_finite_reaches_only_who_attends_it(kb, bad, where, dtype, dn, dr, dv):
    c = Case(kb, dtype, [150, 70, 260, 1, 3], [300, 70, 260, 200, 3], 3, dn, dr, dv, seed=4)
    t = [280, 20, 130, 199, 1]  # a key row, or the query row that sits at it
    for b, x in enumerate(t):
        if where == "q":
            c.q[c.q0[b] + x - (c.kl[b] - c.ql[b]), 1, 5] = bad
        elif where == "pe":
            c.pe[c.k0[b] + x, 3] = bad
        else:
            getattr(c, where)[c.k0[b] + x, 1, 9] = bad
    c.run()
    assert int(c.err) == 0
    out, q, v = c.out.cpu(), c.q.double().cpu(), c.v.double().cpu()
    key = torch.cat((c.k.double().cpu(), c.pe.double().cpu()[:, None].expand(-1, 3, -1)), -1)
    for b, x in enumerate(t):
        first = c.kl[b] - c.ql[b]
        for p in sorted({first, x - 2, x - 1, x, x + 1, c.kl[b] - 1} & set(range(first, c.kl[b]))):
            keys = slice(c.k0[b], c.k0[b] + p + 1)
            w, bound = R.attend(q[c.q0[b] + p - first], key[keys], v[keys], c.scale, c.dt)
            got = out[c.q0[b] + p - first]
            hit = torch.tensor([h == 1 or where == "pe" for h in range(3)]) & (p == x if where == "q" else p >= x)
            R.check(got[~hit], w[~hit], bound[~hit], f"request {b} position {p}")
            if math.isnan(bad):
                assert bool(got[hit].isnan().any(-1).all())


def test_values_that_are_not_finite_in_every_tile(kb):
    """More such tiles than SMs, several to each: rows before the value are right, rows from it on are not finite."""
    c = Case(kb, "bf16", [130] * 20, [130] * 20, 64, 128, 64, 128, seed=6)
    at = [(29 * b + 40) % 127 + 1 for b in range(20)]
    for b in range(20):
        c.v[c.k0[b] + at[b], :, 3 * b] = float("nan") if b % 2 else float("inf")
    c.run()
    c.run()
    assert int(c.err) == 0
    out, q, v = c.out.cpu(), c.q.double().cpu(), c.v.double().cpu()
    key = torch.cat((c.k.double().cpu(), c.pe.double().cpu()[:, None].expand(-1, 64, -1)), -1)
    for b in range(20):
        rows = out[c.q0[b]:c.q0[b + 1]]
        assert bool(rows[:at[b]].isfinite().all()) and not bool(rows[at[b]:].isfinite().all(-1).any())
        for j in {0, at[b] - 1}:
            keys = slice(c.k0[b], c.k0[b] + j + 1)
            w, bound = R.attend(q[c.q0[b] + j], key[keys], v[keys], c.scale, c.dt)
            R.check(rows[j], w, bound, f"request {b} query {j}")


def test_strides(kb):
    """Heads before tokens, odd token strides, and rows that do not start on 16 bytes."""
    a = Case(kb, "bf16", [70, 130], [100, 130], 4, 128, 64, 128, seed=2)
    a.run()
    a.verify()
    want = a.out.clone()
    one = torch.zeros_like(a.k[:, :1]).expand(-1, 4, -1)  # one key part for all heads, by a head stride of zero
    a.k = one
    a.run()
    a.verify()
    a = Case(kb, "bf16", [70, 130], [100, 130], 4, 128, 64, 128, seed=2)
    a.run()
    for f in (lambda t: t.transpose(0, 1).contiguous().transpose(0, 1),
              lambda t: torch.nn.functional.pad(t, (0, 8))[..., :t.shape[-1]],
              lambda t: torch.nn.functional.pad(t, (3, 2))[..., 3:3 + t.shape[-1]]):
        c = Case(kb, "bf16", [70, 130], [100, 130], 4, 128, 64, 128, seed=2)
        c.q, c.k, c.v = f(c.q), f(c.k), f(c.v)
        c.pe = f(c.pe[:, None])[:, 0]
        c.run()
        c.verify()
    assert torch.equal(a.out, want)


def test_bad_offsets_skip_their_request(kb):
    for dn, dr, dv in ((128, 64, 128), (32, 16, 32)):
        for which, what in ((0, [0, 40, 20, 100]), (0, [0, -3, 70, 100]), (0, [0, 40, 70, 101]), (1, [0, 40, 90, 131]),
                            (1, [0, 40, 30, 130])):
            c = Case(kb, "bf16", [40, 30, 30], [40, 50, 40], 2, dn, dr, dv, seed=4)
            (c.qs if which == 0 else c.ks).copy_(torch.tensor(what, dtype=torch.int32))
            c.run()
            assert int(c.err) == kb.KVP_ERR_BAD_INDEX
        c = Case(kb, "bf16", [40, 30, 30], [40, 50, 40], 2, dn, dr, dv, seed=4)
        c.max_q = 35  # the first request has more rows
        c.run()
        assert int(c.err) == kb.KVP_ERR_BAD_INDEX
        assert bool((c.out[:40] == 5.0).all())
        c.verify(only=[1, 2])
        c = Case(kb, "bf16", [40, 30, 30], [40, 50, 40], 2, dn, dr, dv, seed=4)
        c.ks.copy_(torch.tensor([0, 40, 60, 130], dtype=torch.int32))  # 30 queries on 20 keys
        c.k0 = [0, 40, 60]
        c.kl = [40, 20, 70]
        c.run()
        assert int(c.err) == kb.KVP_ERR_BAD_INDEX
        assert bool((c.out[40:70] == 5.0).all())
        c.verify(only=[0, 2])


def test_stream_and_graph(kb):
    c = Case(kb, "bf16", [200, 64], [333, 64], 4, 128, 64, 128, seed=5)
    c.run()
    c.verify()
    want = c.out.clone()
    s = torch.cuda.Stream()
    c.out.fill_(5.0)
    torch.cuda.synchronize()
    c.run(stream=s)
    assert torch.equal(c.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kb.latent_prefill_attention(c.q, c.k, c.pe, c.v, c.qs, c.ks, c.max_q, c.scale, c.out, error_word=c.err)
    c.out.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_large_scores_and_late_maximum(kb):
    c = Case(kb, "bf16", [150], [400], 2, 128, 64, 128, seed=6)
    ramp = torch.linspace(0.01, 8.0, 400, device=DEV)[:, None, None]
    c.k.copy_((c.q[149:150, :, :128].float() * ramp).to(c.dt))
    c.run()
    c.verify()


def test_refusals(kb):
    c = Case(kb, "bf16", [10], [20], 2, 128, 64, 128)
    call = lambda q=c.q, k=c.k, pe=c.pe, v=c.v, qs=c.qs, ks=c.ks, out=c.out, scale=1.0, max_q=10: (  # noqa: E731
        kb.latent_prefill_attention(q, k, pe, v, qs, ks, max_q, scale, out))
    for kw in (dict(q=c.q.half()), dict(k=c.k.float()), dict(qs=c.qs.long()), dict(out=c.out.float())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(pe=None), dict(q=c.q[..., :150]), dict(k=c.k[:, :1]), dict(v=c.v[:19]), dict(out=c.out[:9]),
               dict(ks=torch.cat((c.ks, c.ks))), dict(pe=c.pe[:19]), dict(k=c.k[..., ::2])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(kb.KvpError):
        call(scale=float("nan"))
    with pytest.raises(kb.KvpError):
        call(max_q=-1)
    assert bool((c.out == 5.0).all())


def test_both_forms_agree_on_a_paged_prompt(kb):
    """A prompt through the latent cache: rows stored in pages and read back, the expanded form of the projected rows
    against the absorbed form, W_K moved to the query and W_V to the output."""
    from paged_decode_attention_store_gb300.engine import PagedLatentCache

    H, dn, dr, dc, dv, n = 4, 128, 64, 512, 128, 150
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    cache = PagedLatentCache(64, 16, dc, dr, 2, max_requests=4)
    rope = kb.RotaryPlan(dr, layout="interleaved", device=DEV)
    wk, wv = rnd(H, dn, dc) / math.sqrt(dc), rnd(H, dv, dc) / math.sqrt(dc)
    cache.new(1)
    loc = cache.append([1] * n)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    latent, k_pe = rnd(n, dc).bfloat16(), rnd(n, dr).bfloat16()
    q_nope, q_pe = rnd(n, H, dn).bfloat16(), rnd(n, H, dr).bfloat16()
    q = torch.empty((1, n, H, dc + dr), dtype=torch.bfloat16, device=DEV)
    q[0, ..., :dc] = torch.einsum("nhd,hdc->nhc", q_nope.float(), wk).bfloat16()
    cache.store(1, q_pe, latent, k_pe, pos, loc, rope, q[0])
    scale = 1.0 / math.sqrt(dn + dr)
    out = torch.empty((1, n, H, dc), dtype=torch.bfloat16, device=DEV)
    cache.attend(1, q, torch.tensor([n], dtype=torch.int32, device=DEV), 0, scale, out,
                 table_rows=torch.tensor([1], dtype=torch.int32, device=DEV))
    absorbed = torch.einsum("nhc,hvc->nhv", out[0].float(), wv)
    rows, start = cache.rows(1, [1])
    assert torch.equal(rows[:, :dc], latent) and start.tolist() == [0, n]
    k = torch.einsum("nc,hdc->nhd", rows[:, :dc].float(), wk).bfloat16()
    v = torch.einsum("nc,hvc->nhv", rows[:, :dc].float(), wv).bfloat16()
    ex = torch.empty((n, H, dv), dtype=torch.bfloat16, device=DEV)
    kb.latent_prefill_attention(torch.cat((q_nope, q[0, ..., dc:]), -1), k, rows[:, dc:], v, start, start, n, scale, ex)
    cache.check()
    # both sides carry a handful of bf16 roundings (q or k projected, weights, output: each 2^-8 of its operand at
    # most); a score of size s is moved by 2^-8 sqrt(s^2 / W) ~ 2^-8 each, so 2 % of the output's size holds both
    d = (ex.float() - absorbed).norm() / absorbed.norm()
    assert d < 0.02, float(d)


def test_latent_cache_steps(kb):
    """Prompt chunk, decode steps with a window, fork with copy-on-write, rewind: the engine's step against rows kept
    by the test."""
    from paged_decode_attention_store_gb300.engine import PagedLatentCache

    H, dc, dr, layers = 8, 512, 64, 2
    W = dc + dr
    g = torch.Generator().manual_seed(5)
    cache = PagedLatentCache(96, 16, dc, dr, layers, max_requests=6, table_mode="raw", max_seq_len=512)
    rope = kb.RotaryPlan(dr, device=DEV)
    theta = R.thetas(dr)
    kept = {}
    scale = W ** -0.5

    def step(rids, C, window=0, sinks=0):
        B = len(rids)
        rnd = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)  # noqa: E731
        q = [rnd(B, C, H, W) for _ in range(layers)]
        q_pe = [rnd(B, C, H, dr) for _ in range(layers)]
        lat, pe = [rnd(B * C, dc) for _ in range(layers)], [rnd(B * C, dr) for _ in range(layers)]
        out = [torch.empty((B, C, H, dc), dtype=torch.bfloat16, device=DEV) for _ in range(layers)]
        base = [int(cache.lengths[r]) for r in rids]
        cache.step(rids, q, q_pe, lat, pe, rope, out, window, scale, sinks=sinks)
        cache.check()
        for i, r in enumerate(rids):
            pos = torch.arange(base[i], base[i] + C, dtype=torch.int32)
            for layer in range(layers):
                turned, _ = R.rotate(pe[layer][i * C:(i + 1) * C, None], pos, theta, "half")
                new = torch.cat((lat[layer][i * C:(i + 1) * C].cpu(), turned[:, 0].to(torch.bfloat16)), -1)
                kept[r, layer] = torch.cat((kept.get((r, layer), torch.empty((0, W), dtype=torch.bfloat16)), new))
                for j in {0, C - 1}:
                    p = base[i] + j
                    x = kept[r, layer][R.span(p, window, sinks)].double()
                    w, bound = R.attend(q[layer][i, j].double().cpu(), x, x[:, :dc], scale, torch.bfloat16)
                    # the stored key part may round to the other neighbour (2^-8 of an entry); 64 of them move a
                    # score by at most that times its size, and the weights by as much
                    slack = 2.0 ** -7 * (q[layer][i, j, :, dc:].double().cpu().abs() @ x[:, dc:].abs().T).amax() * scale
                    R.check(out[layer][i, j], w, bound + 2 * slack * x[:, :dc].abs().amax(0), f"request {r} query {j}")

    for r in (0, 3):
        cache.new(r)
    step([0, 3], 37)
    step([3, 0], 1)
    step([0], 20)
    cache.fork(3, 1)
    for layer in range(layers):
        kept[1, layer] = kept[3, layer].clone()
    step([1, 3], 1)
    assert cache.last_copies == 1
    step([0, 1, 3], 5)
    cache.rewind(1, 3)
    for layer in range(layers):
        kept[1, layer] = kept[1, layer][:-3]
    step([1], 2)
    for _ in range(20):
        step([0, 1, 3], 1, window=24, sinks=2)
    for what in ("decode_step", "verify_step", "prefill_step"):
        with pytest.raises(TypeError):
            getattr(cache, what)([0], [torch.empty((1, 1, H, W), device=DEV)], None, None, None, 0, 1.0)
    lengths = cache.lengths.copy()
    for rids in ([1, 1], [1]):  # a request twice, and fewer requests than queries
        with pytest.raises(ValueError):
            cache.step(rids, [torch.empty((2, 1, H, W), device=DEV)], None, None, None, rope, None, 0, scale)
    with pytest.raises(ValueError):
        cache.rows(0, [1])  # the window's steps have released its first pages
    assert kb.kvp_sync_error(cache.pool) == 0 and (cache.lengths == lengths).all()
    cache.new(4)
    slots = cache.append([4] * 20)  # the rows of a prompt, without queries
    lat, pe = torch.randn((20, dc), generator=g).bfloat16().to(DEV), torch.zeros((20, dr)).bfloat16().to(DEV)
    cache.store(1, None, lat, pe, torch.arange(20, dtype=torch.int32, device=DEV), slots, rope, None)
    rows, start = cache.rows(1, [4])
    assert torch.equal(rows, torch.cat((lat, pe), -1)) and start.tolist() == [0, 20]


def test_values_that_are_not_finite_give_the_same_bits(kb):
    """Whichever SM takes a tile, and whether it has met such values before: tiles with and without them, several to
    each SM, come out the same in every call."""
    c = Case(kb, "bf16", [700, 130, 260, 40] * 5, [900, 130, 515, 40] * 5, 24, 128, 64, 128, seed=11)
    for b in range(0, 20, 3):
        for t in range(b % 7, c.kl[b], 97):
            c.v[c.k0[b] + t, (b + t) % 24, t % 128] = float("nan") if t % 2 else float("inf")
    c.run()
    first = c.out.clone()
    assert int(c.err) == 0 and not bool(first.isfinite().all())
    for _ in range(15):
        c.out.fill_(5.0)
        c.run()
        assert int(c.err) == 0 and torch.equal(first.view(torch.int16), c.out.view(torch.int16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,dn,dr,dv", [("bf16", 128, 64, 128), ("bf16", 64, 32, 64), ("f32", 128, 64, 128)])
def test_a_value_that_is_not_finite_reaches_its_entry_alone(kb, bad, dtype, dn, dr, dv):
    """Of the head it is in, for the queries that attend it, wherever in their keys it lies; all else is the formula's."""
    H = 3
    c = Case(kb, dtype, [150, 70, 260, 1, 3], [300, 70, 260, 200, 3], H, dn, dr, dv, seed=8)
    entries = {}  # (request, head) -> (key, entry) that are not finite
    for b, keys in enumerate([(40, 160, 280), (20, 61), (0, 127, 128, 130, 255), (3, 199), (1,)]):
        for i, t in enumerate(keys):
            h, d = i % 2, (37 * i + 9) % dv
            c.v[c.k0[b] + t, h, d] = bad
            entries.setdefault((b, h), []).append((t, d))
    for _ in range(2):
        c.out.fill_(5.0)
        c.run()
        assert int(c.err) == 0
        out, q, v = c.out.cpu(), c.q.double().cpu(), c.v.double().cpu()
        v[~v.isfinite()] = 0.0
        key = torch.cat((c.k.double().cpu(), c.pe.double().cpu()[:, None].expand(-1, H, -1)), -1)
        for b in range(len(c.ql)):
            first = c.kl[b] - c.ql[b]
            near = {t + x for h in range(H) for t, _ in entries.get((b, h), []) for x in (-1, 0, 1)}
            for p in sorted((near | {first, c.kl[b] - 1}) & set(range(first, c.kl[b]))):
                keys = slice(c.k0[b], c.k0[b] + p + 1)
                w, bound = R.attend(q[c.q0[b] + p - first], key[keys], v[keys], c.scale, c.dt)
                hit = torch.zeros((H, dv), dtype=torch.bool)
                for h in range(H):
                    for t, d in entries.get((b, h), []):
                        hit[h, d] |= t <= p
                got = out[c.q0[b] + p - first]
                assert not bool(got[hit].isfinite().any()), f"request {b} position {p}"
                R.check(got[~hit], w[~hit], bound[~hit], f"request {b} position {p}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_value_that_is_not_finite_under_a_score_of_minus_infinity(kb, dtype):
    """A weight of zero does not keep it from its entry, as the formula has it, in whatever order the keys come."""
    for t in (0, 5, 140, 149):
        c = Case(kb, dtype, [150], [150], 2, 128, 64, 128, seed=9)
        c.q[:, 1, 4] = 1.0
        c.k[t, 1, 4] = -float("inf")
        c.v[t, 1, 7] = float("inf")
        c.run()
        hit = torch.zeros((150, 2, 128), dtype=torch.bool)
        hit[t:, 1, 7] = True
        assert not bool(c.out.cpu()[hit].isfinite().any()) and bool(c.out.cpu()[~hit].isfinite().all())


def test_a_long_prompt_among_very_many_requests(kb):
    """1.05e9 tiles of queries of which 128 times 65 have rows: the others take 3 s to come by, longer than any wait but
    the one for the next tile may be."""
    B, H, L, T = 2 ** 17, 128, 8192, 8192 + 7
    g = torch.Generator(device=DEV).manual_seed(3)

    def heads(width):  # overlapping heads, eight entries apart: small inputs
        flat = torch.randn(T * (8 * H + width) + width, generator=g, device=DEV).bfloat16()
        return flat.as_strided((T, H, width), (8 * H + width, 8, 1))

    q, k, v = heads(192), heads(128), heads(128)
    pe = torch.randn((T, 64), generator=g, device=DEV).bfloat16()
    out = torch.full((T, H, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    start = torch.zeros(B + 1, dtype=torch.int32)
    start[B // 3 + 1:] = L
    start[B:] = T
    start, err = start.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    kb.latent_prefill_attention(q, k, pe, v, start, start, L, 192 ** -0.5, out, error_word=err)
    assert int(err) == 0
    for first, n in ((0, L), (L, 7)):
        for j in {0, n // 2, n - 1}:
            keys = slice(first, first + j + 1)
            key = torch.cat((k[keys].double().cpu(), pe[keys].double().cpu()[:, None].expand(-1, H, -1)), -1)[:, ::37]
            w, bound = R.attend(q[first + j, ::37].double().cpu(), key, v[keys, ::37].double().cpu(), 192 ** -0.5,
                                torch.bfloat16)
            R.check(out[first + j, ::37], w, bound, f"query {first + j}")


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "pe"])
@pytest.mark.parametrize("dtype,dn,dr,dv", [("bf16", 128, 64, 128), ("bf16", 64, 32, 64), ("f32", 128, 64, 128)])
def test_an_infinite_key_counts_by_its_score(kb, bad, where, dtype, dn, dr, dv):
    """Minus infinity weighs nothing, plus infinity makes the head's output NaN; a query with that key alone gets zeros."""
    H = 3
    c = Case(kb, dtype, [150, 200, 1], [300, 200, 1], H, dn, dr, dv, seed=12)
    t = [200, 64, 0]
    q, v = c.q.double().cpu(), c.v.double().cpu()
    for b, x in enumerate(t):
        if where == "k":
            c.k[c.k0[b] + x, 1, 5] = bad
        else:
            c.pe[c.k0[b] + x, 5] = bad
    c.run()
    assert int(c.err) == 0
    out = c.out.cpu()
    key = torch.cat((c.k.double().cpu(), c.pe.double().cpu()[:, None].expand(-1, H, -1)), -1)
    seen = set()
    for b, x in enumerate(t):
        first = c.kl[b] - c.ql[b]
        for p in range(max(first, x), min(x + 40, c.kl[b])):
            for h in range(H) if where == "pe" else (1,):
                met = q[c.q0[b] + p - first, h, 5 if where == "k" else dn + 5] * bad
                got = out[c.q0[b] + p - first, h]
                seen.add((float(met), p == 0))
                if met > 0:
                    assert bool(got.isnan().all())
                    continue
                keep = [c.k0[b] + i for i in range(p + 1) if i != x]
                if not keep:
                    assert bool((got == 0).all())
                    continue
                w, bound = R.attend(q[c.q0[b] + p - first, h:h + 1], key[keep][:, h:h + 1], v[keep][:, h:h + 1], c.scale, c.dt)
                R.check(got[None], w, bound, f"request {b} position {p} head {h}")
    assert {s for s, _ in seen} == {float("inf"), -float("inf")}
