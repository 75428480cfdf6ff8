"""Calls of more than 64 (token, head) columns a KV head that are not the chunk kernel's: their weights are fp16, as those of
fewer columns, and their bound is fp16's."""

import pytest
import torch

import fp4_reference as F
import operator_reference as R
from test_gpu_fp4_attention import Case, kb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,C,H,hkv,D,window,sinks", [
    ([300, 411], 20, 32, 8, 128, 0, 0),     # the decode kernel: fewer CTAs than SMs
    ([300, 411], 32, 32, 8, 128, 0, 0),
    ([300, 411], 130, 24, 8, 128, 0, 0),    # the tile kernel
    ([300, 411], 130, 32, 8, 64, 0, 0),
    ([300, 411], 70, 8, 2, 256, 0, 0),
    ([300, 411], 130, 12, 4, 128, 200, 100),
])
def test_weights_are_fp16(kb, lens, C, H, hkv, D, window, sinks):  # noqa: F811
    c = Case(kb, "bf16", lens, C, H, hkv, D, 16, seed=C + D, gk=0.5, gv=2.0)
    c.run(window, sinks)
    G, out = H // hkv, c.out.cpu()
    for b, L in enumerate(lens):
        for j in (0, C // 3, C - 1):
            sl = torch.tensor([c.slots[b][t] for t in R.span(L - C + j, window, sinks)])
            for h in range(hkv):
                at = slice(h * G, (h + 1) * G)
                w, bound = F.attend(c.q[b, j, at].double().cpu(), c.k[sl, h], c.v[sl, h], c.scale, c.dt, torch.float16)
                R.check(out[b, j, at], w, bound, f"request {b} query {j} head {h}")
