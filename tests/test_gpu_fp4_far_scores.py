"""Scores past fp32's range, in every kernel: minus infinity weighs nothing, and a query all of whose scores are gets zeros;
plus infinity makes the head's output NaN."""

import pytest
import torch

import operator_reference as R
from test_gpu_fp4_attention import Case, kb  # noqa: F401
from test_gpu_fp4_decode import bounded, rewrite

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,C,H,hkv,D,most", [
    ("bf16", 1, 32, 8, 128, 1000), ("bf16", 4, 32, 8, 128, 1000), ("bf16", 1, 32, 8, 128, 256), ("bf16", 140, 32, 8, 128, 333),
    ("bf16", 140, 24, 8, 128, 333), ("bf16", 4, 8, 2, 64, 333), ("bf16", 70, 8, 2, 256, 333), ("f32", 1, 32, 8, 128, 333),
    ("f32", 40, 8, 2, 64, 333)])
def test_scores_past_the_range(kb, dtype, C, H, hkv, D, most):  # noqa: F811
    lens = [240, 200] if most == 256 else [333, 200]
    c = bounded(Case(kb, dtype, lens, C, H, hkv, D, 16, seed=3), most)
    k, v = (torch.randn(333, D, generator=torch.Generator().manual_seed(i)) for i in (4, 5))
    k[:, 0] = -2688.0
    k[::3, 0] = 0.0
    rewrite(c, k, v)
    c.q[:, :, 0] = 0
    c.q[:, :, 0, 0] = 2.0 ** 126    # - 2^137 with most keys, 0 with the others
    c.q[:, :, 1] = 0
    c.q[:, :, 1, 0] = -2.0 ** 126   # + 2^137 with most keys
    c.run()
    assert kb.kvp_sync_error(c.pool) == 0
    out = c.out.cpu()
    vals = c.v[:, 0]
    for b in range(2):
        for j in sorted({0, C // 2, C - 1}):
            seen = torch.tensor(c.slots[b][:lens[b] - C + j + 1])
            level = vals[seen[::3]]
            # the weights are one and zero: the fp32 sums and the result's rounding are left
            bound = R.u(c.dt) * level.mean(0).abs() + 2 * (len(seen) + 16) * R.U32 * level.abs().amax(0)
            R.check(out[b, j, 0], level.mean(0), bound, f"request {b} query {j}")
            assert bool(out[b, j, 1].isnan().all())
    k[:, 0] = -2688.0
    rewrite(c, k, v)
    c.run()
    assert bool((c.out[:, :, 0] == 0).all()) and bool(c.out[:, :, 1].isnan().all()) and not bool(c.out[:, :, 2:].isnan().any())
