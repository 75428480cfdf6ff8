"""The four-bit store of keys whose turned entries pass fp32's range: codes and scales are those of the 64-bit formula."""

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from test_gpu_fp4_store import DEV, DT, check_rows, kb, make_pool, slots_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("attn", [1.0, 1.25, 2.0 ** 60])
@pytest.mark.parametrize("aligned", [True, False])
def test_turned_entries_past_the_range(kb, dtype, layout, attn, aligned):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    n, hkv, D, rot = 40, 4, 64, 32
    most = torch.finfo(DT[dtype]).max
    x = torch.randn((n, 2 * hkv, D), generator=g)
    x[:, :hkv, ::7] = torch.where(torch.rand((n, hkv, 10), generator=g) < 0.5, most, -most)
    x[5:9, :hkv] = most           # a sum of two, and a difference that is none
    x[9:12, :hkv, ::2] = -most
    x[12, :hkv, 3], x[13, :hkv, 20] = float("inf"), float("nan")
    x = x.to(DT[dtype])
    g0, pages = 2.0 ** 64, 5
    pool = make_pool(kb, pages, 16, hkv, D, dtype, ks=g0)
    buf = torch.zeros(x.numel() + 1, dtype=x.dtype, device=DEV)
    kv = buf[0 if aligned else 1:][:x.numel()].view(x.shape)
    kv.copy_(x)
    pos = torch.randint(0, 1 << 16, (1, n), generator=g, dtype=torch.int32)
    loc = slots_of(n, pages * 16, g)
    kb.rotary_store_fp4(pool, 0, None, kv[:, :hkv], kv[:, hkv:], pos[0].to(DEV), loc.to(DEV),
                        kb.RotaryPlan(rot, layout=layout, attn_factor=attn, device=DEV), None)
    assert kb.kvp_sync_error(pool) == 0
    want, _ = F.rotate_axes(x[:, :hkv], pos, R.thetas(rot), [0] * (rot // 2), layout, attn)
    good = torch.isfinite(want).unflatten(-1, (-1, 16)).all(-1)
    assert bool(good[[i for i in range(n) if i not in (12, 13)]].all()) and not bool(good[12:14].all())
    check_rows(pool, loc, want, x[:, hkv:].double(), g0, 1.0)
