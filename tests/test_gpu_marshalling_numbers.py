"""Numbers that no C type holds: the C++ marshalling leaves them to Python's refusal, and nothing is launched."""

import pytest
import torch

from test_gpu_marshalling import DEV, kb, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [dict(scale=10 ** 400), dict(scale=-10 ** 400), dict(layer=1 << 32), dict(layer=-1 << 70),
                                 dict(sinks=1 << 40), dict(max_context=-1 << 40)])
def test_numbers_past_their_range(kb, bad):  # noqa: F811
    pool = kb.kv_fp4_pool_create(8, 16, 2, 64, kb.KVP_BF16, 1, device=DEV, zero=True)
    q = rnd(2, 1, 8, 64)
    out = torch.full_like(q, 5.0)
    table, lens = torch.zeros((2, 8), dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    ws = kb.alloc_fp4_workspace(pool, 2, 1, 8, 128, device=DEV)
    a = dict(dict(layer=0, window=0, sinks=0, scale=0.1, max_context=None), **bad)

    def attend():
        kb.paged_fp4_attention(pool, a["layer"], q, table, kb.KVP_BLOCK_TABLE, lens, a["window"], a["scale"], out, ws,
                               sinks=a["sinks"], max_context=a["max_context"])
    with pytest.raises((OverflowError, kb.KvpError)):
        attend()
    torch.cuda.synchronize()
    assert bool((out == 5.0).all()) and kb.kvp_sync_error(pool) == 0
    a = dict(layer=0, window=1 << 40, sinks=3, scale=0.1, max_context=1 << 40)  # no window, any context
    attend()
    assert kb.kvp_sync_error(pool) == 0 and not bool((out == 5.0).any())


@pytest.mark.parametrize("layer", [1 << 32, 1 << 70, -1 << 32])
def test_layers_past_their_range(kb, layer):  # noqa: F811
    pool = kb.kv_fp4_pool_create(8, 16, 2, 64, kb.KVP_BF16, 1, device=DEV, zero=True)
    x, i = rnd(3, 2, 64), torch.arange(3, dtype=torch.int32, device=DEV)
    with pytest.raises(OverflowError):
        kb.store_cache_fp4(pool, layer, x, x, i)
    with pytest.raises(OverflowError):
        kb.load_cache_fp4(pool, layer, i, x, x)
    assert not bool(pool.codes.any())
