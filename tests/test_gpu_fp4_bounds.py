"""What bounds a four-bit cache's calls beside a long request: the step's own lengths, and a workspace of limited size."""

import pytest
import torch

import operator_reference as R
from test_gpu_fp4_attention import DEV, Case
from test_gpu_fp4_cache import Steps, kb  # noqa: F401
from test_gpu_fp4_decode import bounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("host", [None, "prefill_step", "verify_step"])
def test_steps_beside_a_long_request(kb, monkeypatch, host):  # noqa: F811
    s = Steps(kb, "bf16", 32, 8, 128, 16, "block")
    for r in (1, 4, 5):
        s.cache.new(r)
    s.cache.append([5] * 700)
    given, attend = [], kb.paged_fp4_attention
    monkeypatch.setattr(kb, "paged_fp4_attention", lambda *a, **kw: given.append(kw["max_context"]) or attend(*a, **kw))
    s.step([1, 4], 100, host=host)
    s.step([4, 1], 30, host=host)
    s.step([4], 130, host=host)
    assert given == [256, 256, 256, 256, 512, 512]


LIMIT = 1 << 32  # of a chunk's workspace


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("most,hkv", [(262144, 8), (400000, 8), (1 << 19, 4), ((1 << 20) + 1, 8)])
def test_chunks_in_a_limited_workspace(kb, most, hkv, rows):  # noqa: F811
    """Bounds of which 4 GiB hold three requests, two, two (4 heads), and none: the requests go through it in groups, the
    last by another kernel. An invalid request and a NaN in a later group."""
    lens, q_lens = [300, 411, 177, 500, 440], [140, 1, 140, 139, 77]
    c = Case(kb, "bf16", lens, 140, 4 * hkv, hkv, 128, 16, seed=5)
    order = [3, 0, 4, 1, 2] if rows else list(range(5))
    if rows:
        moved = c.table.clone()
        for b, r in enumerate(order):
            moved[r] = c.table[b]
        c.table = moved
    table_rows = torch.tensor(order, dtype=torch.int32, device=DEV) if rows else None
    c.clens[3] = most + 1
    slot = c.slots[4][-1]  # seen by the last query alone
    c.pool.scales[0, slot // 16, hkv - 1, slot % 16, 1, 2] = 0x7F
    c.run(q_lens=q_lens, table_rows=table_rows)
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    want = c.out.clone()
    assert kb.paged_fp4_attention_workspace_size(c.pool, 5, 140, c.H, most) == LIMIT
    bounded(c, most, 0xFF)
    assert c.ws.numel() == LIMIT
    c.out.fill_(5.0)
    c.run(q_lens=q_lens, table_rows=table_rows)
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    assert bool((c.out[3] == 0).all())
    nan = c.out[4].isnan().cpu()
    assert bool(nan[76, -4:, 32:48].all()) and int(nan.sum()) == 64
    if most <= 1 << 19:
        assert torch.equal(c.out.nan_to_num(7.0), want.nan_to_num(7.0))  # in groups or at once: the same bits
    c.verify(only=[0, 1, 2], q_lens=q_lens)
    w, bound = c.want(4, 40, 77)
    R.check(c.out[4, 40].cpu(), w, bound)


def test_a_workspace_does_not_shrink(kb):  # noqa: F811
    """A workspace that serves a call serves its smaller ones."""
    pool = kb.kv_fp4_pool_create(8, 16, 8, 128, kb.KVP_BF16, 1, device=DEV)
    size = lambda B, C, most: kb.paged_fp4_attention_workspace_size(pool, B, C, 32, most)  # noqa: E731
    for C in (1, 20, 32, 140, 512):
        for steps in ([(B, 100000) for B in (1, 2, 5, 10, 11, 40, 64, 1000)],
                      [(7, most) for most in (1, 300, 5000, 149000, 150000, 500000, 1 << 20, 1 << 21, (1 << 31) - 1)]):
            sizes = [size(B, C, most) for B, most in steps]
            assert sizes == sorted(sizes) and sizes[-1] <= LIMIT


def test_few_columns_of_many_long_contexts(kb):  # noqa: F811
    """Groups that would leave SMs idle: all requests at once, by a kernel without such rows."""
    c = Case(kb, "bf16", [300, 411, 177, 500], 44, 4, 1, 128, 16, seed=5)
    bounded(c, 6_000_000, 0xFF)
    assert c.ws.numel() == LIMIT
    c.run()
    c.verify()


def test_groups_captured_and_replayed(kb):  # noqa: F811
    """Requests that go through the workspace in groups, over a raw table, in a graph that is replayed with other lengths."""
    c = bounded(Case(kb, "bf16", [300, 411, 177, 500], 140, 32, 8, 128, 16, raw=True, seed=5), 400000)
    want = c.run().clone()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        kb.paged_fp4_attention(c.pool, 0, c.q, c.table, kb.KVP_RAW_LOCATIONS, c.clens, 0, c.scale, c.out, c.ws, max_context=c.most)
    for lens in ([300, 411, 177, 500], [150, 411, 140, 260], [300, 411, 177, 500]):
        c.clens.copy_(torch.tensor(lens))
        c.out.fill_(5.0)
        c.lens = lens
        g.replay()
        torch.cuda.synchronize()
        assert kb.kvp_sync_error(c.pool) == 0
        c.verify(few=True)
    assert torch.equal(c.out, want)
