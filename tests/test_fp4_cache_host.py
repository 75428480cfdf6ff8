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
