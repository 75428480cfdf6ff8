"""PagedFp4Cache: steps, prompts, forks, windows and host tensors against the 64-bit formulas."""

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from libbuild import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FEW = 64


@pytest.fixture(scope="module")
def kb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_built()


class Steps:
    """A cache, what its steps were given, and the checks of what they left."""

    def __init__(self, kb, dtype, H, hkv, D, P, table_mode, sections=None, layers=2, gk=1.0, gv=0.5):
        from paged_decode_attention_store_gb300.engine import PagedFp4Cache

        self.g = torch.Generator().manual_seed(D + P)
        self.kb, self.dt, self.H, self.hkv, self.D, self.layers, self.gk, self.gv = kb, DT[dtype], H, hkv, D, layers, gk, gv
        self.cache = PagedFp4Cache(1200 // P + 60, P, hkv, D, layers, dtype=dtype, max_requests=6, table_mode=table_mode,
                                   max_seq_len=768, k_scale=gk, v_scale=gv)
        self.sections = sections
        self.plan = kb.RotaryPlan(D, device=DEV, sections=sections)
        self.of_pair = kb.pair_axes(sections) if sections else [0] * (D // 2)
        self.theta, self.scale = R.thetas(D), D ** -0.5
        self.want = {}  # (request, layer) -> codes' values of K and V

    def rnd(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dt).to(DEV)

    def step(self, rids, C, window=0, sinks=0, rope=True, positions=None, host=None):
        B, H, hkv, D = len(rids), self.H, self.hkv, self.D
        q = [self.rnd(B, C, H, D) for _ in range(self.layers)]
        given = [x.clone() for x in q]
        k, v = ([self.rnd(B * C, hkv, D) for _ in range(self.layers)] for _ in range(2))
        out = [torch.empty((B, C, H, D), dtype=self.dt, device=DEV) for _ in range(self.layers)]
        base = [int(self.cache.lengths[r]) for r in rids]
        places = torch.cat([torch.arange(b, b + C) for b in base])
        axes = self.plan.axes
        pos = places.expand(axes, -1) if positions is None else positions.cpu().view(axes, -1)
        if host:
            pin = lambda ts: [t.cpu().pin_memory() for t in ts]  # noqa: E731
            back = pin(out)
            getattr(self.cache, host)(rids, pin(q), pin(k), pin(v), back, window, self.scale, sinks=sinks)
            out = back
        else:
            self.cache.step(rids, q, k, v, self.plan if rope else None, out, window, self.scale, sinks=sinks,
                            positions=positions)
        self.cache.check()
        turn = rope and not host
        for layer in range(self.layers):
            kk = F.rotate_axes(k[layer], pos, self.theta, self.of_pair, "half")[0] if turn else k[layer].double().cpu()
            if turn:
                w, bound = F.rotate_axes(given[layer].view(B * C, H, D), pos, self.theta, self.of_pair, "half")
                R.check(q[layer].view(B * C, H, D), w, bound + R.u(self.dt) * (w.abs() + bound), "queries")
            new = [F.values(*F.quantise(x, g), g) for x, g in ((kk, self.gk), (v[layer].double().cpu(), self.gv))]
            for i, r in enumerate(rids):
                old = self.want.get((r, layer))
                mine = [x[i * C:(i + 1) * C] for x in new]
                self.want[r, layer] = mine if old is None else [torch.cat(p) for p in zip(old, mine)]
                K, V = self.want[r, layer]
                for j in sorted({0, C // 2, C - 1}):
                    sl = torch.tensor(R.span(base[i] + j, window, sinks))
                    G = H // hkv
                    for h in (0, hkv - 1):
                        w, bound = F.attend(q[layer][i, j, h * G:(h + 1) * G].double().cpu(), K[sl, h], V[sl, h], self.scale,
                                            self.dt, torch.float16 if C * G <= FEW else torch.bfloat16)
                        R.check(out[layer][i, j, h * G:(h + 1) * G], w, bound, f"request {r} query {j} head {h}")

    def check_rows(self, rids):
        for layer in range(self.layers):
            k, v, start = self.cache.rows(layer, rids)
            want = [torch.cat([self.want[r, layer][p] for r in rids]) for p in (0, 1)]
            assert torch.equal(k.double().cpu(), want[0]) and torch.equal(v.double().cpu(), want[1])
            assert start.tolist()[-1] == k.shape[0]


CASES = [
    ("bf16", 32, 8, 128, 16, "block", None),
    ("bf16", 8, 2, 128, 1, "raw", (16, 24, 24)),
    ("bf16", 8, 8, 128, 4, "block", (32, 32)),
    ("bf16", 4, 4, 64, 16, "raw", None),
    ("f32", 8, 4, 32, 4, "block", (4, 6, 6)),
]


@pytest.mark.parametrize("dtype,H,hkv,D,P,table,sections", CASES)
def test_prompts_steps_forks_and_rewinds(kb, dtype, H, hkv, D, P, table, sections):
    s = Steps(kb, dtype, H, hkv, D, P, table, sections)
    for r in (0, 3):
        s.cache.new(r)
    s.step([0, 3], 37)
    s.step([3, 0], 1)
    s.step([0], 120)
    s.cache.fork(3, 1)
    for layer in range(s.layers):
        s.want[1, layer] = s.want[3, layer]
    s.step([1, 3], 1)       # the shared tail page is copied, scales and all
    s.step([3, 1, 0], 5)
    s.cache.rewind(1, 3)
    for layer in range(s.layers):
        s.want[1, layer] = [x[:-3] for x in s.want[1, layer]]
    s.step([1, 0, 3], 1)
    s.check_rows([3, 0, 1])
    if sections:
        s.step([0, 1], 3, positions=torch.randint(0, 900, (len(sections), 6), generator=s.g, dtype=torch.int32).to(DEV))
    s.step([3], 4, rope=False)
    s.check_rows([1, 3, 0])


@pytest.mark.parametrize("sinks", [0, 3])
def test_a_window_releases_pages(kb, sinks):
    s = Steps(kb, "bf16", 32, 8, 128, 16, "block")
    for r in (0, 2):
        s.cache.new(r)
    s.step([0, 2], 90, window=50, sinks=sinks)
    used = s.cache.host.used()
    for _ in range(20):
        s.step([2, 0], 1, window=50, sinks=sinks)
    s.step([0, 2], 6, window=50, sinks=sinks)
    assert s.cache.host.used() <= used + 2
    with pytest.raises(ValueError, match="released"):
        s.cache.rows(0, [0])


def test_steps_of_host_tensors(kb):
    s = Steps(kb, "bf16", 32, 8, 128, 16, "block")
    for r in (1, 4):
        s.cache.new(r)
    s.step([1, 4], 100, host="prefill_step")
    s.step([4, 1], 4, host="verify_step")
    s.check_rows([1, 4])


def test_a_refused_step_leaves_the_cache(kb):
    s = Steps(kb, "bf16", 8, 2, 128, 16, "block")
    s.cache.new(0)
    s.step([0], 20)
    before = (s.cache.lengths.copy(), s.cache.host.used(), s.cache.host.block_row(0))
    q, o = [s.rnd(1, 3, 8, 128) for _ in range(2)], [s.rnd(1, 3, 8, 128) for _ in range(2)]
    k = [s.rnd(3, 2, 128) for _ in range(2)]
    for bad in (dict(v=[k[0], k[1][:2]]), dict(rids=[0, 0]), dict(rope=kb.RotaryPlan(256, device=DEV)),
                dict(positions=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(window=5, sinks=5)):
        a = dict(rids=[0], q=q, k=k, v=k, rope=s.plan, out=o, window=0, scale=1.0)
        a.update(bad)
        with pytest.raises((ValueError, kb.KvpError)):
            s.cache.step(**a)
    assert (s.cache.lengths == before[0]).all() and (s.cache.host.used(), s.cache.host.block_row(0)) == before[1:]
    s.step([0], 1)
    with pytest.raises(TypeError):
        s.cache.decode_step([0], None, None, None, None, 0, 1.0)
    with pytest.raises(TypeError):
        s.cache.store_and_attend(0)


def test_the_example_runs(kb):
    """The example of a four-bit cache in README.md, as written."""
    import os
    import re

    from libbuild import ROOT

    text = open(os.path.join(ROOT, "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "PagedFp4Cache(" in c][0]
    env = {"torch": torch, "RotaryPlan": kb.RotaryPlan}
    exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(env["out"][0].float()).all()) and env["out"][0].shape == (1, 1, 32, 128)
    assert env["keys"].shape == env["values"].shape == (271, 8, 128) and bool(torch.isfinite(env["keys"].float()).all())
    env["cache"].check()
