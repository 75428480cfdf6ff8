"""The argument marshalling in C++ and Python's own way make the same calls, and Python's refusals stand."""

import pytest
import torch

from libbuild import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Python:
    """Marshalling that leaves every call to Python."""

    @staticmethod
    def leave(*args):
        return None

    rotary = load = attend = leave


class Counted:
    """The marshalling in C++; ``done`` counts the calls it made."""

    def __init__(self, native):
        self.native, self.done = native, 0

    def __getattr__(self, name):
        def call(*args):
            code = getattr(self.native, name)(*args)
            self.done += code is not None
            return code
        return call


@pytest.fixture(scope="module")
def kb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_built()


def rnd(*shape, dtype=torch.bfloat16, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


KINDS = [(kind, part) for kind in ("cache", "axes", "latent", "fp4") for part in ("all", "queries", "rows")] + [("as they are", "rows")]


@pytest.mark.parametrize("kind,part", KINDS)
@pytest.mark.parametrize("n", [0, 1, 5])
@pytest.mark.parametrize("strided", [False, True])
def test_rotary_stores(kb, monkeypatch, kind, n, part, strided):
    D, H, hkv, dc = 64, 6, 2, 32
    sections = (10, 10, 12) if kind in ("axes", "fp4") else None
    plan = kb.RotaryPlan(D, sections=sections, attn_factor=1.5)
    positions = torch.randint(0, 99, (3, n + 4), dtype=torch.int32, generator=torch.Generator().manual_seed(2)).to(DEV)[:, :n]
    if not sections:
        positions = positions[0].contiguous()
    loc = torch.randperm(48)[:n].to(torch.int32).to(DEV)
    wide = rnd(n, 2 * (H + 2 * hkv), D)
    heads = wide[:, :H + 2 * hkv] if strided else wide[:, :H + 2 * hkv].contiguous()
    q, k, v = heads[:, :H], heads[:, H:H + hkv], heads[:, H + hkv:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    results = []
    native = Counted(kb._native())
    for way in (native, Python()):
        monkeypatch.setattr(kb, "_native", lambda way=way: way)
        q_out = torch.zeros((n, H, D), dtype=torch.bfloat16, device=DEV)
        a = dict(q=q if part != "rows" else None, out_loc=loc if part != "queries" else None, positions=positions,
                 layer=0, rope=plan)
        if kind == "latent":
            buf = torch.zeros((1, 3, 16, dc + D), dtype=torch.bfloat16, device=DEV)
            pool = kb.LatentPool(buf, dc, kb.KVP_BF16)
            kb.rotary_store_latent(pool, 0, a["q"], v[:, 0, :dc] if part != "queries" else None,
                                   k[:, 0] if part != "queries" else None, positions, a["out_loc"], plan,
                                   q_out if part != "rows" else None)
            state = buf
        else:
            kv = (k, v) if part != "queries" else (None, None)
            if kind == "as they are":
                pool = kb.kv_fp4_pool_create(3, 16, hkv, D, kb.KVP_BF16, 1, device=DEV, zero=True)
                kb.store_cache_fp4(pool, 0, *kv, loc)
                state = torch.cat((pool.codes.flatten(), pool.scales.flatten()))
            elif kind == "fp4":
                pool = kb.kv_fp4_pool_create(3, 16, hkv, D, kb.KVP_BF16, 1, device=DEV, zero=True)
                kb.rotary_store_fp4(pool, 0, a["q"], *kv, positions, a["out_loc"], plan, q_out if part != "rows" else None)
                state = torch.cat((pool.codes.flatten(), pool.scales.flatten()))
            else:
                buf = torch.zeros((2, 1, 3, 16, hkv, D), dtype=torch.bfloat16, device=DEV)
                pool = kb.Pool(buf, 16, kb.KVP_BF16)
                kb.rotary_store_cache(pool, 0, a["q"], *kv, positions, a["out_loc"], plan, q_out if part != "rows" else None)
                state = buf
        assert kb.kvp_sync_error(pool) == 0
        results.append((q_out, state))
    assert native.done == 1
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert n == 0 or part == "rows" or bool(results[0][0].any())
    assert n == 0 or part == "queries" or bool(results[0][1].any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("raw", [False, True])
def test_rows_back_and_attention(kb, monkeypatch, dtype, raw):
    dt, kdt = (torch.bfloat16, kb.KVP_BF16) if dtype == "bf16" else (torch.float32, kb.KVP_F32)
    pool = kb.kv_fp4_pool_create(8, 16, 2, 64, kdt, 1, device=DEV, zero=True)
    slots = torch.arange(100, dtype=torch.int32, device=DEV)
    kb.store_cache_fp4(pool, 0, rnd(100, 2, 64, dtype=dt), rnd(100, 2, 64, dtype=dt, seed=3), slots)
    table = (torch.arange(128) if raw else torch.arange(8)).int().to(DEV).expand(2, -1).contiguous()
    mode = kb.KVP_RAW_LOCATIONS if raw else kb.KVP_BLOCK_TABLE
    lens, ql, rows = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([100, 40], [3, 2], [1, 0]))
    q = rnd(2, 3, 8, 64, dtype=dt)
    ws = kb.alloc_fp4_workspace(pool, 2, 3, 8, 128, device=DEV)
    side = torch.cuda.Stream()
    results = []
    native = Counted(kb._native())
    for way in (native, Python()):
        monkeypatch.setattr(kb, "_native", lambda way=way: way)
        got = []
        for kw in (dict(), dict(q_lens=ql), dict(table_rows=rows, max_context=100), dict(window=20, sinks=2), dict(stream=side),
                   dict(stream=side.cuda_stream), dict(window=None), dict(scale=1), dict(max_context=1 << 40)):
            out = torch.zeros_like(q)
            side.wait_stream(torch.cuda.current_stream())
            kw = dict(dict(window=0, scale=0.1), **kw)
            window, scale = kw.pop("window"), kw.pop("scale")
            kb.paged_fp4_attention(pool, 0, q, table, mode, lens, window, scale, out, ws, **kw)
            torch.cuda.synchronize()
            got.append(out)
        k, v = (torch.zeros((100, 2, 64), dtype=dt, device=DEV) for _ in range(2))
        kb.load_cache_fp4(pool, 0, slots.flip(0), k, v)
        assert kb.kvp_sync_error(pool) == 0
        results.append(got + [k, v])
    assert native.done == 10
    assert all(torch.equal(x, y) for x, y in zip(*results)) and all(bool(x.any()) for x in results[0])


def test_refusals_are_pythons(kb):
    pool = kb.kv_fp4_pool_create(8, 16, 2, 64, kb.KVP_BF16, 1, device=DEV, zero=True)
    q, i32 = rnd(2, 1, 8, 64), dict(dtype=torch.int32, device=DEV)
    table, lens = torch.zeros((2, 8), **i32), torch.ones(2, **i32)
    ws = kb.alloc_fp4_workspace(pool, 2, 1, 8, 128, device=DEV)
    good = dict(q=q, table=table, lens=lens, out=torch.zeros_like(q), ws=ws, layer=0, window=0, sinks=0, scale=0.1)

    def attend(**kw):
        a = dict(good, **kw)
        kb.paged_fp4_attention(pool, a["layer"], a["q"], a["table"], kb.KVP_BLOCK_TABLE, a["lens"], a["window"], a["scale"],
                               a["out"], a["ws"], sinks=a["sinks"])

    attend()
    for bad, error in ((dict(q=q.cpu()), TypeError), (dict(q=q.float()), TypeError), (dict(q=q[:, 0]), ValueError),
                       (dict(q=q.transpose(1, 2)), ValueError), (dict(table=table.long()), TypeError),
                       (dict(table=table[:, ::2]), ValueError), (dict(lens=lens[:1]), ValueError), (dict(out=q[:1]), ValueError),
                       (dict(ws=ws.cpu()), TypeError), (dict(ws=ws[:16]), kb.KvpError), (dict(layer=1), kb.KvpError),
                       (dict(window=4, sinks=4), kb.KvpError), (dict(scale=float("nan")), kb.KvpError)):
        with pytest.raises(error):
            attend(**bad)
    k = rnd(4, 2, 64)
    plan, pos = kb.RotaryPlan(64), torch.arange(4, **i32)
    for bad, error in ((dict(k=k[:3]), ValueError), (dict(k=k.float()), TypeError), (dict(positions=pos.long()), TypeError),
                       (dict(positions=pos[:3]), ValueError), (dict(out_loc=pos[::2]), ValueError), (dict(v=None), ValueError),
                       (dict(q=rnd(4, 3, 64)), TypeError), (dict(rope=kb.RotaryPlan(128)), ValueError)):
        a = dict(dict(q=None, k=k, v=k, positions=pos, out_loc=pos, rope=plan), **bad)
        with pytest.raises(error):
            kb.rotary_store_fp4(pool, 0, a["q"], a["k"], a["v"], a["positions"], a["out_loc"], a["rope"], None)
    with pytest.raises(ValueError):
        kb.load_cache_fp4(pool, 0, pos, k[:3], k)
    torch.cuda.synchronize()
    assert kb.kvp_sync_error(pool) == 0
