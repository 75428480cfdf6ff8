"""Positions of several axes on latent pools of either type, aligned and not, and axes that are none on a four-bit pool."""

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from test_gpu_rotary_axes import DEV, DT, kb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,dc,dr,rot,layout,sections,pad", [
    (45, 64, 32, 32, "half", (4, 12), 0), (45, 64, 32, 32, "interleaved", (4, 6, 6), 0), (45, 64, 32, 32, "half", (4, 12), 1),
    (45, 60, 12, 10, "interleaved", (2, 3), 0), (9100, 64, 32, 32, "interleaved", (16, 0), 0)])
def test_latent_rows(kb, dtype, n, dc, dr, rot, layout, sections, pad):  # noqa: F811
    g = torch.Generator().manual_seed(n + rot)
    H, pages, dt = 4, -(-n // 16) + 1, DT[dtype]
    buf = torch.zeros((1, pages, 16, dc + dr), dtype=dt, device=DEV)
    pool = kb.LatentPool(buf, dc, kb.KVP_BF16 if dtype == "bf16" else kb.KVP_F32)
    down = torch.randn((n, dc + dr + pad), generator=g).to(dt)  # with a pad: rows that do not start on 16 bytes
    qp = torch.randn((n, H, dr), generator=g).to(dt)
    loc = torch.randperm(16 * pages, generator=g)[:n].to(torch.int32)
    pos = torch.randint(-4096, 4096, (len(sections), n), generator=g, dtype=torch.int32)
    q = torch.zeros((n, H, dc + dr), dtype=dt, device=DEV)
    d = down.to(DEV)
    plan = kb.RotaryPlan(rot, device=DEV, layout=layout, sections=sections, interleave=True, attn_factor=0.75)
    kb.rotary_store_latent(pool, 0, qp.to(DEV), d[:, :dc], d[:, dc:dc + dr], pos.to(DEV), loc.to(DEV), plan, q[..., dc:])
    assert kb.kvp_sync_error(pool) == 0
    of_pair, rows = kb.pair_axes(sections, True), buf.view(-1, dc + dr)[loc.to(DEV).long()]
    for got, part in ((q[..., dc:], qp), (rows[:, None, dc:], down[:, None, dc:dc + dr])):
        w, bound = F.rotate_axes(part, pos, R.thetas(rot), of_pair, layout, 0.75)
        R.check(got, w, bound + R.u(dt) * (w.abs() + bound))
    assert torch.equal(rows[:, :dc], d[:, :dc]) and not bool(q[..., :dc].any())


@pytest.mark.parametrize("pad", [0, 1])
def test_an_axis_that_is_none_counts_as_the_first(kb, pad):  # noqa: F811
    n, hkv, D = 30, 2, 64
    pools = [kb.kv_fp4_pool_create(2, 16, hkv, D, kb.KVP_BF16, 1, device=DEV, zero=True) for _ in range(2)]
    x = torch.randn(n * hkv * D + 1, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)[pad:][:n * hkv * D]
    x = x.view(n, hkv, D)
    pos = torch.stack((torch.arange(n), 7 * torch.arange(n))).int().to(DEV)
    for pool, axis in zip(pools, (2, 0)):
        plan = kb.RotaryPlan(D, device=DEV, sections=(16, 16))
        plan.pair_axis[20] = axis
        kb.rotary_store_fp4(pool, 0, None, x, x, pos, torch.arange(n, dtype=torch.int32, device=DEV), plan, None)
        assert kb.kvp_sync_error(pool) == (kb.KVP_ERR_BAD_INDEX if axis else 0)
    assert torch.equal(pools[0].codes, pools[1].codes) and torch.equal(pools[0].scales, pools[1].scales)
    assert bool(pools[0].codes.any())
