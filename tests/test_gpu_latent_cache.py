"""PagedLatentCache.step against the 64-bit formulas: where each query and each row stands."""

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


class Steps:
    """A cache, what its steps were given, and the checks of what they left."""

    def __init__(self, kb, dtype, dc, dr, H, P, table_mode, layout, scaling, layers=2):
        from paged_decode_attention_store_gb300.engine import PagedLatentCache

        self.g = torch.Generator().manual_seed(dc + P)
        self.kb, self.dt, self.dc, self.dr, self.H, self.P, self.layers, self.layout = kb, DT[dtype], dc, dr, H, P, layers, layout
        self.cache = PagedLatentCache(400 // P + 60, P, dc, dr, layers, dtype=dtype, max_requests=6, table_mode=table_mode,
                                      max_seq_len=384)
        factor = 1.0 if scaling == "none" else 8.0
        self.plan = kb.RotaryPlan(dr, layout=layout, scaling=scaling, factor=factor, attn_factor=1.25, device=DEV)
        self.theta = R.thetas(dr, scaling=scaling, factor=factor)
        self.scale = (dc + dr) ** -0.5
        self.given = {}  # (request, layer) -> latents and key parts as given

    def rnd(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dt).to(DEV)

    def rotated(self, x, pos):
        """(want, bound) of x [n, heads, dr] at ``pos``; a neighbouring position is further off than the bound."""
        want, bound = R.rotate(x, pos, self.theta, self.layout, self.plan.attn_factor)
        bound = bound + R.u(self.dt) * (want.abs() + bound)
        for by in (-1, 1):
            other, _ = R.rotate(x, pos + by, self.theta, self.layout, self.plan.attn_factor)
            assert bool(((other - want).abs() > 2 * bound).flatten(1).any(1).all())
        return want, bound

    def stored(self, layer, rid, n):
        """Rows 0 .. n - 1 of a request, found through the table here."""
        t = torch.arange(n)
        row = self.cache.table[rid].cpu().long()
        slots = row[t] if self.cache.raw else row[t // self.P] * self.P + t % self.P
        return self.cache.kv[layer].reshape(-1, self.dc + self.dr)[slots.to(DEV)]

    def step(self, rids, C, window=0, sinks=0):
        B, H, dc, dr = len(rids), self.H, self.dc, self.dr
        q = [self.rnd(B, C, H, dc + dr) for _ in range(self.layers)]
        absorbed = [x[..., :dc].clone() for x in q]
        q_pe = [self.rnd(B, C, H, dr) for _ in range(self.layers)]
        latent, k_pe = ([self.rnd(B * C, w) for _ in range(self.layers)] for w in (dc, dr))
        out = [torch.empty((B, C, H, dc), dtype=self.dt, device=DEV) for _ in range(self.layers)]
        base = [int(self.cache.lengths[r]) for r in rids]
        self.cache.step(rids, q, q_pe, latent, k_pe, self.plan, out, window, self.scale, sinks=sinks)
        self.cache.check()
        for layer in range(self.layers):
            assert torch.equal(q[layer][..., :dc], absorbed[layer])
            for i, r in enumerate(rids):
                pos = torch.arange(base[i], base[i] + C)
                want, bound = self.rotated(q_pe[layer][i], pos)
                R.check(q[layer][i, ..., dc:], want, bound, f"queries of request {r}")
                new = slice(i * C, (i + 1) * C)
                a, b = self.given.get((r, layer), (latent[layer][:0], k_pe[layer][:0]))
                self.given[r, layer] = torch.cat((a, latent[layer][new])), torch.cat((b, k_pe[layer][new]))
                if window:
                    continue  # this step has released the pages that its window leaves
                x = self.rows(layer, r)
                for j in sorted({0, C // 2, C - 1}):
                    keys = x[:base[i] + j + 1].double().cpu()
                    w, bound = R.attend(q[layer][i, j].double().cpu(), keys, keys[:, :dc], self.scale, self.dt)
                    R.check(out[layer][i, j], w, bound, f"request {r} query {j}")
        return q, out, base

    def rows(self, layer, rid):
        """The stored rows of a request, each checked against what was given at its position."""
        latent, k_pe = self.given[rid, layer]
        x = self.stored(layer, rid, len(latent))
        assert torch.equal(x[:, :self.dc], latent)
        want, bound = self.rotated(k_pe[:, None], torch.arange(len(latent)))
        R.check(x[:, None, self.dc:], want, bound, f"rows of request {rid}")
        return x


CASES = [
    # dtype, dc, dr, H, P, table, layout, scaling
    ("bf16", 512, 64, 8, 16, "block", "half", "none"),
    ("bf16", 512, 64, 24, 1, "raw", "interleaved", "by_parts"),
    ("bf16", 512, 64, 80, 4, "raw", "half", "linear"),
    ("bf16", 128, 32, 3, 16, "block", "interleaved", "ntk"),
    ("f32", 64, 16, 4, 4, "block", "half", "none"),
]


@pytest.mark.parametrize("dtype,dc,dr,H,P,table,layout,scaling", CASES)
def test_steps_put_queries_and_rows_at_their_positions(kb, dtype, dc, dr, H, P, table, layout, scaling):
    """Prompts, decode and verify steps, forks, rewinds and steps in another order of the requests."""
    s = Steps(kb, dtype, dc, dr, H, P, table, layout, scaling)
    for r in (0, 3):
        s.cache.new(r)
    s.step([0, 3], 37)
    s.step([3, 0], 1)
    s.step([0], 20)
    s.cache.fork(3, 1)
    for layer in range(s.layers):
        s.given[1, layer] = s.given[3, layer]
    s.step([1, 3], 1)
    s.step([3, 1, 0], 5)
    s.cache.rewind(1, 3)
    for layer in range(s.layers):
        s.given[1, layer] = tuple(t[:-3] for t in s.given[1, layer])
    s.step([1], 2)
    s.step([0, 1, 3], 1)


def test_windowed_steps_put_queries_at_their_positions(kb):
    """With a window and sinks, over rows that the window has left: the outputs from the rows as given."""
    s = Steps(kb, "bf16", 512, 64, 8, 16, "block", "half", "none", layers=1)
    s.cache.new(2)
    window, sinks = 40, 3
    for C in (90, 1, 4, 1, 1, 3) + (1,) * 20:
        q, out, base = s.step([2], C, window, sinks)
        latent, k_pe = s.given[2, 0]
        turned, _ = R.rotate(k_pe[:, None], torch.arange(len(latent)), s.theta, s.layout, s.plan.attn_factor)
        for j in sorted({0, C - 1}):
            span = R.span(base[0] + j, window, sinks)
            keys = torch.cat((latent.double().cpu(), turned[:, 0]), 1)[span]
            w, bound = R.attend(q[0][0, j].double().cpu(), keys, keys[:, :512], s.scale, s.dt)
            # these keys are not rounded as the stored ones are: an entry by u of itself, a score by u sum |q||k| at most,
            # which moves a weight by as much relative, and the sum of weights as well
            off = R.u(s.dt) * (q[0][0, j, :, 512:].double().cpu().abs() @ keys[:, 512:].abs().T).amax(-1) * s.scale
            weights = torch.softmax(q[0][0, j].double().cpu() @ keys.T * s.scale, -1)
            R.check(out[0][0, j], w, bound + (2 * torch.expm1(off))[:, None] * (weights @ keys[:, :512].abs()), f"query {j}")


def test_a_step_that_is_refused_leaves_the_cache_as_it_was(kb):
    s = Steps(kb, "bf16", 512, 64, 8, 16, "block", "half", "none")
    s.cache.new(0)
    s.cache.new(1)
    s.step([0, 1], 30)
    before, free = s.cache.lengths.copy(), s.cache.host.free_list()
    table = s.cache.table.clone()
    B, C, H, dc, dr = 2, 5, s.H, s.dc, s.dr
    good = dict(q=s.rnd(B, C, H, dc + dr), q_pe=s.rnd(B, C, H, dr), latent=s.rnd(B * C, dc), k_pe=s.rnd(B * C, dr),
                out=torch.empty((B, C, H, dc), dtype=s.dt, device=DEV), window=0, sinks=0, scale=s.scale, plan=s.plan)

    def call(**kw):
        a = {**good, **kw}
        s.cache.step([0, 1], *([a[x]] * 2 for x in ("q", "q_pe", "latent", "k_pe")), a["plan"], [a["out"]] * 2, a["window"],
                     a["scale"], sinks=a["sinks"])

    for kw in (dict(latent=s.rnd(B * C - 1, dc)), dict(k_pe=s.rnd(B * C, dr + 8)), dict(latent=good["latent"].float()),
               dict(out=good["out"][..., :8]), dict(window=4, sinks=4), dict(scale=float("nan")),
               dict(plan=kb.RotaryPlan(2 * dr, device=DEV)), dict(plan=kb.RotaryPlan(dr, device="cpu"))):
        with pytest.raises((ValueError, TypeError, kb.KvpError)):
            call(**kw)
        assert (s.cache.lengths == before).all() and s.cache.host.free_list() == free
        assert [s.cache.host.length(r)[0] for r in (0, 1)] == [30, 30]
    torch.cuda.synchronize()
    assert torch.equal(s.cache.table, table)
    s.step([0, 1], C)
    s.step([1, 0], 1)


def test_rows_of_requests_without_tokens(kb):
    """They have none, alone or among others, and leave no error behind."""
    s = Steps(kb, "bf16", 512, 64, 8, 16, "block", "half", "none")
    for r in range(4):
        s.cache.new(r)
    for rids in ([], [0], [0, 3]):
        rows, start = s.cache.rows(0, rids)
        assert rows.shape == (0, 576) and rows.dtype == s.dt and start.tolist() == [0] * (len(rids) + 1)
    s.step([1, 3], 20)
    rows, start = s.cache.rows(1, [0, 3, 2, 1])
    assert start.tolist() == [0, 0, 20, 20, 40]
    assert torch.equal(rows, torch.cat((s.rows(1, 3), s.rows(1, 1))))
    s.cache.check()
