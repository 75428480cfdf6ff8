"""The rotary stores of K/V and latent pools refuse a call without positions before any launch; a four-bit pool takes rows as
they are without them."""

import ctypes

import pytest
import torch

from libbuild import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def kb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_built()


@pytest.mark.parametrize("kind", ["cache", "cache_axes", "latent", "latent without rope", "latent_axes", "fp4"])
@pytest.mark.parametrize("aligned", [True, False])
def test_no_positions(kb, kind, aligned):
    n, hkv, D = 5, 2, 64
    if kind.startswith("latent"):
        pool = kb.LatentPool(torch.zeros((1, 4, 16, 2 * D), dtype=torch.bfloat16, device=DEV), 2 * D if "without" in kind else D,
                             kb.KVP_BF16)
        state = pool.kv_buffer
    elif kind == "fp4":
        pool = kb.kv_fp4_pool_create(4, 16, hkv, D, kb.KVP_BF16, 1, device=DEV, zero=True)
        state = pool.codes
    else:
        pool = kb.kv_pool_create(4, 16, hkv, D, kb.KVP_BF16, 1, torch.zeros((2, 1, 4, 16, hkv, D), dtype=torch.bfloat16, device=DEV))
        state = pool.kv_buffer
    rows = torch.ones(n * hkv * D + 1, dtype=torch.bfloat16, device=DEV)[0 if aligned else 1:][:n * hkv * D]
    loc = torch.arange(n, dtype=torch.int32, device=DEV)
    name = {"cache": "rotary_store_cache", "cache_axes": "rotary_store_cache_axes", "latent_axes": "rotary_store_latent_axes",
            "fp4": "rotary_store_fp4"}.get(kind, "rotary_store_latent")
    axes = "axes" in kind or kind == "fp4"
    p, stride = ctypes.c_void_p(rows.data_ptr()), hkv * D
    where = (None, 0) if axes else (None,)
    plan = (None, None, 1, 0) if axes else (None, 0)
    code = getattr(kb.lib(), name)(pool.handle, 0, None, 0, 0, 0, p, stride, p, stride, *where, ctypes.c_void_p(loc.data_ptr()), n,
                                   *plan, 0, 1.0, None, 0, 0, None)
    torch.cuda.synchronize()
    assert code == (kb.KVP_OK if kind == "fp4" else kb.KVP_ERR_INVALID_ARG)
    assert bool(state.any()) == (kind == "fp4") and kb.kvp_sync_error(pool) == 0


def test_rows_as_they_are_are_for_four_bits(kb):
    """The Python call without a plan and positions."""
    pool = kb.kv_pool_create(4, 16, 2, 64, kb.KVP_BF16, 1, device=DEV)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    loc = torch.arange(3, dtype=torch.int32, device=DEV)
    with pytest.raises(kb.KvpError):
        kb.rotary_store_cache(pool, 0, None, k, k, None, loc, None, None)
