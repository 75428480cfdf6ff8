"""A block whose scale is the NaN of either sign (0x7f, 0xff) reaches the queries that attend it and no others, in every
kernel."""

import pytest
import torch

import operator_reference as R
from test_gpu_fp4_attention import Case, kb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nan", [0x7F, 0xFF])
@pytest.mark.parametrize("dtype,C,H,hkv,D,most", [
    ("bf16", 4, 32, 8, 128, 1000), ("bf16", 7, 8, 1, 128, 1000), ("bf16", 4, 8, 8, 128, 256), ("bf16", 140, 32, 8, 128, 333),
    ("bf16", 140, 24, 8, 128, 333), ("bf16", 4, 8, 2, 64, 333), ("bf16", 50, 2, 1, 256, 333), ("f32", 4, 32, 8, 128, 333)])
def test_either_nan(kb, nan, dtype, C, H, hkv, D, most):  # noqa: F811
    lens = [180, 240] if most == 256 else [180, 333]
    c = Case(kb, dtype, lens, C, H, hkv, D, 16, seed=7)
    c.most = most
    c.ws = kb.alloc_fp4_workspace(c.pool, 2, C, H, most)
    cut, block = C // 2, D // 16 - 2
    kt, vt = lens[0] - cut, lens[1] - cut  # the last ``cut`` tokens' first row
    for slot, head, part, at in ((c.slots[0][kt], 0, 0, 1), (c.slots[1][vt], hkv - 1, 1, block)):
        c.pool.scales[0, slot // 16, head, slot % 16, part, at] = nan
    c.run()
    assert kb.kvp_sync_error(c.pool) == 0
    G, out, lo = H // hkv, c.out.float().cpu(), 16 * block
    for j in range(C):
        sees = j >= C - cut
        assert bool(out[0, j, :G].isnan().all()) == sees and bool(out[0, j, :G].isnan().any()) == sees, j
        assert not bool(out[0, j, G:].isnan().any())
        last = out[1, j, H - G:]
        assert bool(last[:, lo:lo + 16].isnan().all()) == sees and bool(last[:, lo:lo + 16].isnan().any()) == sees, j
        assert not bool(last[:, :lo].isnan().any()) and not bool(last[:, lo + 16:].isnan().any())
        assert not bool(out[1, j, :H - G].isnan().any())
    for b in range(2):
        w, bound = c.want(b, 0, C)
        R.check(c.out[b, 0].cpu(), w, bound, f"request {b}")
    k, v = (torch.zeros((1, hkv, D), dtype=c.dt, device=c.q.device) for _ in range(2))
    kb.load_cache_fp4(c.pool, 0, torch.tensor([c.slots[1][vt]], dtype=torch.int32, device=k.device), k, v)
    assert bool(v[0, hkv - 1, lo:lo + 16].isnan().all()) and int(v.isnan().sum()) == 16
