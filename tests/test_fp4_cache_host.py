"""PagedFp4Cache's own decisions, without a GPU: its page bookkeeping is real, the pool and the device calls are recorded."""

import types

import numpy as np
import pytest
import torch

from libbuild import ensure_built

H, HKV, D, P, LAYERS = 4, 2, 64, 16, 2


@pytest.fixture
def cache(monkeypatch):
    kb = ensure_built()
    from paged_decode_attention_store_gb300 import engine

    calls = []
    pool = types.SimpleNamespace(codes=None, scales=None, error_word=None, dtype=kb.KVP_BF16, device_index=-1, kv_heads=HKV,
                                 head_dim=D, num_layers=LAYERS)
    monkeypatch.setattr(kb, "kv_fp4_pool_create", lambda *a, **kw: pool)
    monkeypatch.setattr(kb, "paged_fp4_attention_workspace_size", lambda pool, B, C, Hq, most: calls.append(("size", B, most)) or 256)
    for name in ("page_table_write", "copy_pages", "rotary_store_fp4", "store_cache_fp4", "paged_fp4_attention"):
        monkeypatch.setattr(kb, name, lambda *a, _n=name, **kw: calls.append((_n, a, kw)))
    monkeypatch.setattr(engine.PagedKVCache, "_to_device", lambda self, x: torch.from_numpy(np.ascontiguousarray(x, np.int32)))
    c = engine.PagedFp4Cache(2048, P, HKV, D, LAYERS, max_requests=8, max_seq_len=20000, device="cpu")
    c.calls = calls
    return c


def rnd(*shape):
    return [torch.zeros(shape, dtype=torch.bfloat16) for _ in range(LAYERS)]


def plan(kb):
    return kb.RotaryPlan(D, device="cpu")


def attended(c):
    return [(a[2].shape, kw["max_context"]) for n, a, kw in (x for x in c.calls if x[0] == "paged_fp4_attention")]


def step(c, rids, C, **kw):
    B = len(rids)
    a = dict(q=rnd(B, C, H, D), k=rnd(B * C, HKV, D), v=rnd(B * C, HKV, D), rope=plan(ensure_built()), out=rnd(B, C, H, D),
             window=0, scale=0.125)
    a.update(kw)
    c.step(rids, **a)


def test_a_step_is_bounded_by_its_own_requests(cache):
    for r in range(4):
        cache.new(r)
    step(cache, [0], 17000)
    cache.calls.clear()
    step(cache, [1, 2], 200)
    assert attended(cache) == [((2, 200, H, D), 256)] * LAYERS
    assert [x for x in cache.calls if x[0] == "size"] == [("size", 2, 256)]
    cache.calls.clear()
    step(cache, [2, 1, 3], 57)
    assert attended(cache) == [((3, 57, H, D), 512)] * LAYERS  # 257 of one
    cache.calls.clear()
    step(cache, [1, 0], 1)
    assert attended(cache) == [((2, 1, H, D), -(-17001 // 256) * 256)] * LAYERS


def test_verify_and_prefill_take_a_bound(cache):
    for r in (0, 1):
        cache.new(r)
    cache.append([0] * 5000 + [1] * 40)
    q, lens = torch.zeros((1, 3, H, D), dtype=torch.bfloat16), torch.tensor([40], dtype=torch.int32)
    cache.verify(0, q, lens, 0, 0.125, q, max_context=64)
    cache.prefill(0, q, lens, 0, 0.125, q, q_lens=lens, max_context=96)
    cache.prefill(0, q, lens, 0, 0.125, q)  # without one: of the whole cache
    assert [m for _, m in attended(cache)] == [64, 96, 5120]


def bad_steps():
    short = lambda ts: [ts[0], ts[1][:, :1]]  # noqa: E731
    q, k = rnd(1, 3, H, D), rnd(3, HKV, D)
    odd = torch.zeros(3 * H * D + 1, dtype=torch.bfloat16)[1:].view(1, 3, H, D)
    return {
        "q of another shape": dict(q=short(q)), "q of another type": dict(q=[q[0], q[1].float()]),
        "q that is not contiguous": dict(q=[q[0], torch.zeros((1, H, 3, D), dtype=torch.bfloat16).transpose(1, 2)]),
        "q off 16 bytes": dict(q=[q[0], odd]), "q of one layer": dict(q=q[:1]), "q of no tensor": dict(q=[q[0], None]),
        "out of another shape": dict(out=short(q)), "out of another type": dict(out=[q[0].float(), q[1]]),
        "out off 16 bytes": dict(out=[odd, q[1]]), "out of one layer": dict(out=q[:1]),
        "k of fewer tokens": dict(k=[k[0], k[1][:2]]), "v of other heads": dict(v=[k[0], k[1][:, :1]]),
        "v of one layer": dict(v=k[:1]), "k of another type": dict(k=[k[0], k[1].float()]),
        "rows of k apart": dict(k=[k[0], torch.zeros((3, HKV, 2 * D), dtype=torch.bfloat16)[..., ::2]]),
        "scale": dict(scale=float("nan")), "sinks": dict(window=4, sinks=4), "fewer than none": dict(sinks=-1),
        "width": dict(q=rnd(1, 3, H, D // 2), out=rnd(1, 3, H, D // 2)),
    }


@pytest.mark.parametrize("what", bad_steps())
def test_a_refused_step_turns_no_queries(cache, what):
    cache.new(0)
    step(cache, [0], 20)
    cache.calls.clear()
    before = (cache.lengths.copy(), cache.host.used(), cache.host.block_row(0))
    with pytest.raises((ValueError, TypeError, IndexError)):
        step(cache, [0], 3, **bad_steps()[what])
    assert [c[0] for c in cache.calls if c[0] not in ("size", "page_table_write")] == []
    assert (cache.lengths == before[0]).all() and (cache.host.used(), cache.host.block_row(0)) == before[1:]
    step(cache, [0], 3)
    assert len(attended(cache)) == LAYERS


def test_heads_that_do_not_divide(cache, monkeypatch):
    """What the workspace's size refuses is refused before anything else."""
    kb = ensure_built()
    cache.new(0)

    def refuse(*a):
        raise kb.KvpError(kb.KVP_ERR_INVALID_ARG, "paged_fp4_attention_workspace_size")

    monkeypatch.setattr(kb, "paged_fp4_attention_workspace_size", refuse)
    with pytest.raises(kb.KvpError):
        step(cache, [0], 3)
    assert cache.calls == [] and cache.lengths[0] == 0


@pytest.mark.parametrize("what", ["width", "positions", "axes", "factor", "device", "layer"])
def test_a_refused_step_keeps_shared_pages(cache, what):
    """A request that shares its last page: an append would copy it, a refused step does not."""
    kb = ensure_built()
    cache.new(0)
    step(cache, [0], 20)
    cache.fork(0, 1)
    before = (cache.host.used(), cache.host.block_row(0), cache.host.block_row(1), cache.host.refcounts())
    cache.calls.clear()
    elsewhere = plan(kb)
    elsewhere.freqs = types.SimpleNamespace(get_device=lambda: 1, is_cuda=True, device="cuda:1")
    bad = {"width": dict(rope=kb.RotaryPlan(2 * D, device="cpu")), "positions": dict(positions=torch.zeros(2, dtype=torch.int32)),
           "axes": dict(rope=kb.RotaryPlan(D, device="cpu", sections=(16, 16)), positions=torch.zeros(3, dtype=torch.int32)),
           "factor": dict(rope=kb.RotaryPlan(D, device="cpu", attn_factor=float("nan"))), "device": dict(rope=elsewhere),
           "layer": dict(v=[torch.zeros((3, HKV, D), dtype=torch.bfloat16), None])}[what]
    with pytest.raises((ValueError, TypeError)):
        step(cache, [1], 3, **bad)
    assert (cache.host.used(), cache.host.block_row(0), cache.host.block_row(1), cache.host.refcounts()) == before
    assert [x for x in cache.calls if x[0] != "size"] == [] and cache.lengths[1] == 20
    step(cache, [1], 3)
    assert cache.host.used() == before[0] + 1
