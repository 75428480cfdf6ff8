"""paged_fp4_attention at the shapes of neither the decode kernel nor the chunk kernel: other widths, groups that do not
divide 128, negative scales of many queries, fp32; and calls of several host threads."""

import threading

import pytest
import torch

import operator_reference as R
from test_gpu_fp4_attention import DEV, Case, kb  # noqa: F401

pytestmark = pytest.mark.gpu


CASES = [
    # lens, C, H, hkv, D, P, raw, window, sinks
    ([1], 1, 8, 8, 16, 16, False, 0, 0),
    ([1, 63, 64, 65, 128, 129, 1000], 1, 32, 8, 64, 16, False, 0, 0),
    ([33, 500], 1, 16, 16, 48, 16, False, 0, 0),                    # an odd number of blocks
    ([33, 500], 1, 16, 8, 80, 4, True, 0, 0),
    ([33, 500], 1, 32, 4, 96, 24, False, 0, 0),
    ([33, 500], 1, 14, 2, 192, 16, False, 0, 0),
    ([1, 33, 500], 1, 16, 1, 256, 16, False, 0, 0),                 # sixteen columns
    ([33, 500], 1, 17, 1, 256, 1, True, 0, 0),                      # seventeen
    ([4, 66, 700], 4, 32, 8, 64, 16, False, 0, 0),
    ([5, 64, 169], 5, 28, 2, 64, 16, False, 0, 0),                  # seventy columns: two tiles
    ([16, 64, 169], 16, 8, 2, 64, 16, False, 0, 0),                 # sixty-four: one
    ([300, 411], 130, 32, 8, 64, 16, False, 0, 0),
    ([300, 411], 130, 8, 4, 96, 16, False, 0, 0),
    ([70, 411], 70, 8, 4, 256, 16, False, 0, 0),
    ([200, 411], 200, 24, 8, 128, 16, False, 0, 0),                 # three heads a key head
    ([131], 131, 5, 1, 128, 3, True, 0, 0),
    ([3, 64, 100, 1000], 1, 32, 8, 64, 16, False, 50, 0),
    ([40, 64, 100, 1000], 1, 32, 8, 64, 16, False, 70, 40),
    ([40, 64, 1000], 1, 8, 2, 256, 16, False, 130, 65),
    ([300, 411], 130, 16, 4, 64, 4, True, 33, 5),
    ([300, 411], 130, 12, 4, 128, 16, False, 200, 100),
]


@pytest.mark.parametrize("lens,C,H,hkv,D,P,raw,window,sinks", CASES)
def test_attention_is_the_formula(kb, lens, C, H, hkv, D, P, raw, window, sinks):  # noqa: F811
    c = Case(kb, "bf16", lens, C, H, hkv, D, P, raw, seed=C + H + D, gk=2.0, gv=0.25)
    c.run(window, sinks)
    c.verify(window, sinks)
    assert kb.kvp_sync_error(c.pool) == 0


F32 = [
    ([1], 1, 8, 8, 16, 16, False, 0, 0),
    ([1, 31, 32, 33, 63, 64, 65, 129, 1000], 1, 32, 8, 128, 16, False, 0, 0),
    ([33, 500], 1, 16, 16, 48, 16, False, 0, 0),
    ([33, 500], 1, 14, 2, 192, 16, False, 0, 0),                    # seven columns
    ([1, 33, 500], 1, 16, 1, 256, 16, False, 0, 0),                 # sixteen
    ([33, 500], 1, 17, 1, 256, 1, True, 0, 0),                      # seventeen
    ([4, 66, 700], 4, 32, 8, 128, 16, False, 0, 0),
    ([8, 64, 169], 8, 8, 2, 64, 16, False, 0, 0),                   # thirty-two: one tile
    ([9, 64, 169], 9, 8, 2, 64, 16, False, 0, 0),                   # thirty-six: two
    ([130, 211], 130, 12, 4, 128, 16, False, 0, 0),
    ([131], 131, 5, 1, 128, 3, True, 0, 0),
    ([40, 64, 100, 1000], 1, 32, 8, 128, 16, False, 70, 40),
    ([130, 211], 130, 16, 4, 64, 4, True, 33, 5),
    ([30011], 1, 8, 2, 128, 16, False, 0, 0),
]


@pytest.mark.parametrize("lens,C,H,hkv,D,P,raw,window,sinks", F32)
def test_attention_in_fp32(kb, lens, C, H, hkv, D, P, raw, window, sinks):  # noqa: F811
    c = Case(kb, "f32", lens, C, H, hkv, D, P, raw, seed=C + H + D, gk=2.0, gv=0.25)
    first = c.run(window, sinks).clone()
    c.verify(window, sinks, few=True)
    assert kb.kvp_sync_error(c.pool) == 0
    c.run(window, sinks)
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("C", [1, 70])
def test_fp32_bad_requests_holes_and_queries(kb, C):  # noqa: F811
    c = Case(kb, "f32", [200, 100, 220, 170, 250, 300], C, 32, 8, 128, 16, seed=6)
    c.clens.copy_(torch.tensor([200, 0, 100000, 170, 250, 300]))
    c.table[4, 3], c.table[4, 5] = -1, 1 << 30
    c.q[5, 0, 9, 7], c.q[5, 0, 13, 7] = float("nan"), float("inf")
    c.q[5, 0, 3] *= 2.0 ** 60
    c.q[5, 0, 4] *= 2.0 ** -60
    c.q[5, 0, 5] = 0
    rows = torch.tensor([0, 1, 2, 77, 4, 5], dtype=torch.int32, device=DEV)
    c.run(table_rows=rows)
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    assert bool((c.out[1:4] == 0).all())
    c.verify(only=[0])
    w, bound = c.want(5, 0, C)
    bad = c.out[5, 0].cpu().isnan()
    assert bool(bad[[9, 13]].all()) and int(bad.any(-1).sum()) == 2
    keep = [h for h in range(32) if h not in (3, 9, 13)]
    R.check(c.out[5, 0].cpu()[keep], w[keep], bound[keep])
    R.check(c.out[5, 0, 3].cpu(), w[3], 2 * R.u(torch.float32) * w[3].abs() + 1e-30)  # one key has all the weight


@pytest.mark.parametrize("D,H,hkv", [(64, 32, 8), (256, 8, 2), (128, 24, 8)])
def test_ragged_queries(kb, D, H, hkv):  # noqa: F811
    q_lens, lens = [200, 1, 77, 130, 2], [200, 300, 77, 431, 64]
    for window, sinks in ((0, 0), (40, 3)):
        c = Case(kb, "bf16", lens, 200, H, hkv, D, 16, seed=4)
        c.run(window, sinks, q_lens=q_lens)
        c.verify(window, sinks, q_lens=q_lens)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("L", [30, 64, 127, 129, 640, 30011])
def test_one_request_is_shared_by_a_cluster(kb, D, L):  # noqa: F811
    c = Case(kb, "bf16", [L], 1, 8, 2, D, 16, seed=3)
    first = c.run().clone()
    c.verify()
    c.ws.fill_(0x3C)
    c.run()
    assert torch.equal(first, c.out)


def test_more_context_than_there_is(kb):  # noqa: F811
    """A bound far above the lengths: CTAs without a block."""
    c = Case(kb, "bf16", [10, 70, 300], 1, 8, 2, 64, 16, seed=3)
    c.table = torch.cat((c.table, torch.full((3, 4096), -1, dtype=torch.int32, device=DEV)), 1).contiguous()
    c.most = 65536
    c.ws = kb.alloc_fp4_workspace(c.pool, 3, 1, 8, c.most, device=DEV)
    c.run()
    c.verify()


@pytest.mark.parametrize("most", [200, 256, 257, 5000])
@pytest.mark.parametrize("C,H,hkv,raw", [(1, 32, 8, False), (4, 32, 8, False), (1, 16, 1, True), (16, 2, 2, False), (17, 2, 2, True)])
def test_short_contexts_under_any_bound(kb, C, H, hkv, raw, most):  # noqa: F811
    """The bound chooses the kernel, and with more of the same requests their number does."""
    for window, sinks, times in ((0, 0, 1), (0, 0, 20), (40, 3, 1)):
        lens = [L for L in (17, 31, 32, 33, 63, 64, 65, 200) if L >= C] * times
        c = Case(kb, "bf16", lens if C > 1 else lens + [1, 2], C, H, hkv, 128, 1 if raw else 16, raw, seed=C + H)
        c.most = most
        c.ws = kb.alloc_fp4_workspace(c.pool, len(c.lens), C, H, most, device=DEV)
        c.run(window, sinks)
        c.verify(window, sinks, only=range(len(c.lens) - 7, len(c.lens)))
        assert kb.kvp_sync_error(c.pool) == 0


@pytest.mark.parametrize("C,H,hkv", [(1, 32, 8), (4, 32, 8), (140, 32, 8)])
def test_bad_requests_are_zeros_and_recorded(kb, C, H, hkv):  # noqa: F811
    c = Case(kb, "bf16", [200, 1, 220, 170, 250], C, H, hkv, 64, 16, seed=6)
    c.clens.copy_(torch.tensor([200, 0, 100000, 170, 250]))
    rows = torch.tensor([0, 1, 2, 77, 4], dtype=torch.int32, device=DEV)
    c.run(table_rows=rows)
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    assert bool((c.out[1:4] == 0).all())
    c.verify(only=[0, 4])


@pytest.mark.parametrize("C", [1, 140])
def test_holes_are_skipped_and_recorded(kb, C):  # noqa: F811
    c = Case(kb, "bf16", [200, 220], C, 32, 8, 64, 16, seed=6)
    c.table[0, 3] = -1
    c.table[0, 5] = 1 << 30
    c.run()
    assert kb.kvp_sync_error(c.pool) == kb.KVP_ERR_BAD_INDEX
    c.verify(only=[1])


@pytest.mark.parametrize("C,H,hkv,D,dtype", [(1, 32, 8, 64, "bf16"), (4, 32, 8, 64, "bf16"), (140, 32, 8, 64, "bf16"),
                                             (30, 2, 1, 256, "bf16"), (50, 9, 3, 128, "bf16"), (1, 32, 8, 128, "f32"),
                                             (4, 32, 8, 64, "f32"), (50, 9, 3, 128, "f32"), (30, 2, 1, 256, "f32")])
def test_blocks_of_nan_reach_who_attends_them(kb, C, H, hkv, D, dtype):  # noqa: F811
    lens = [180, 333]
    c = Case(kb, dtype, lens, C, H, hkv, D, 16, seed=7)
    cut, block = max(1, C // 2), D // 16 - 2
    kt, vt = c.lens[0] - cut, c.lens[1] - cut
    for slot, head, part, at in ((c.slots[0][kt], 0, 0, 2), (c.slots[1][vt], hkv - 1, 1, block)):
        c.pool.scales[0, slot // 16, head, slot % 16, part, at] = 0x7F
    c.run()
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
        for j in (0, C - cut - 1):
            if 0 <= j < C - cut:
                w, bound = c.want(b, j, C)
                R.check(c.out[b, j].cpu(), w, bound, f"request {b} query {j}")


@pytest.mark.parametrize("C", [1, 40])
def test_queries_of_any_size(kb, C):  # noqa: F811
    c = Case(kb, "bf16", [150, 99], C, 32, 8, 64, 16, seed=9)
    for h, e in ((0, -100), (1, -40), (3, 100)):
        c.q[:, :, h] *= 2.0 ** e
    c.q[:, :, 4] = 0
    c.q[:, :, 5, ::3] *= 2.0 ** -30
    c.q[0, 0, 9, 7] = float("nan")
    c.q[0, 0, 10, 7] = float("inf")
    c.run()
    out = c.out.cpu()
    bad = out.isnan().all(-1)
    assert bool(bad[0, 0, 9]) and bool(bad[0, 0, 10]) and int(out.isnan().any(-1).sum()) == 2
    for b in range(2):
        for j in range(0, C, 7):
            w, bound = c.want(b, j, C)
            keep = [h for h in range(32) if h not in (3, 9, 10)]
            R.check(out[b, j, keep], w[keep], bound[keep])
            R.check(out[b, j, 3], w[3], R.u(torch.bfloat16) * w[3].abs() + 1e-30)  # one key has all the weight


@pytest.mark.parametrize("C,H,hkv,D", [(1, 32, 8, 64), (130, 24, 8, 128), (130, 8, 8, 128)])
def test_scores_that_climb(kb, C, H, hkv, D):  # noqa: F811
    c = Case(kb, "bf16", [700, 300], C, H, hkv, D, 16, seed=10, mag=3.0)
    c.q *= 4
    for scale in (c.scale, -c.scale, 0.0):
        c.scale = scale
        c.run()
        c.verify(few=True)


def test_captured_and_replayed(kb):  # noqa: F811
    c = Case(kb, "bf16", [300, 411], 4, 32, 8, 64, 16, seed=12)
    want = c.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kb.paged_fp4_attention(c.pool, 0, c.q, c.table, kb.KVP_BLOCK_TABLE, c.clens, 0, c.scale, c.out, c.ws,
                               max_context=c.most)
    c.out.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)
    c.clens.copy_(torch.tensor([200, 141]))
    g.replay()
    torch.cuda.synchronize()
    c.lens = [200, 141]
    c.verify()


def test_host_threads_with_other_shapes(kb):  # noqa: F811
    """One pool, four threads with their own streams, workspaces and shapes: each call's result is the one it has alone."""
    c = Case(kb, "bf16", [300, 411, 77], 140, 32, 8, 128, 16, seed=13)
    kind, shapes = kb.KVP_BLOCK_TABLE, (1, 4, 20, 140)
    jobs = []
    for C in shapes:
        q = c.q[:, :C].contiguous()
        ql = torch.tensor([min(C, L) for L in c.lens], dtype=torch.int32, device=DEV)
        jobs.append([C, q, ql, kb.alloc_fp4_workspace(c.pool, 3, C, 32, c.most, device=DEV), torch.cuda.Stream()])
    def call(C, q, ql, ws, out, stream):
        kb.paged_fp4_attention(c.pool, 0, q, c.table, kind, c.clens, 0, c.scale, out, ws, q_lens=ql, stream=stream,
                               max_context=c.most)
    want, got, errors = [], [], []
    for C, q, ql, ws, _ in jobs:
        out = torch.zeros_like(q)
        call(C, q, ql, ws, out, None)
        want.append(out)
        got.append([torch.zeros_like(q) for _ in range(30)])
    torch.cuda.synchronize()

    def work(i):
        try:
            C, q, ql, ws, stream = jobs[i]
            for out in got[i]:
                call(C, q, ql, ws, out, stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for w, outs in zip(want, got):
        for out in outs:
            assert torch.equal(w, out)
