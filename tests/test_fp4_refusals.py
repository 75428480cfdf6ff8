"""Four-bit pools and positions of several axes: what is refused before any launch, and what the plan's host side computes
(CPU only)."""

import ctypes
import types

import pytest
import torch

from libbuild import ensure_built
from test_operator_devices import Library, On, on

B, C, H, D, HKV, N = 2, 1, 4, 64, 2, 3


def test_pools_that_cannot_be():
    kb = ensure_built()
    lib, p, out = kb.lib(), ctypes.c_void_p(256), ctypes.c_void_p()
    null = ctypes.c_void_p()

    def make(pages=4, P=16, hkv=8, d=128, dt=1, layers=2, codes=p, scales=p, ks=None, vs=None, err=p, o=ctypes.byref(out)):
        arr = lambda g: None if g is None else (ctypes.c_float * len(g))(*g)  # noqa: E731
        return lib.kv_fp4_pool_create(pages, P, hkv, d, dt, layers, codes, scales, arr(ks), arr(vs), err, o)

    for kw in (dict(pages=0), dict(P=0), dict(hkv=0), dict(d=0), dict(d=24), dict(d=272), dict(hkv=1, d=64), dict(hkv=3, d=16),
               dict(dt=2), dict(layers=0), dict(codes=null), dict(scales=null), dict(codes=ctypes.c_void_p(8)),
               dict(scales=ctypes.c_void_p(8)), dict(err=null), dict(o=None), dict(pages=1 << 28),
               dict(ks=[1.0, 3.0]), dict(ks=[0.0, 1.0]), dict(vs=[1.0, -2.0]), dict(vs=[float("inf"), 1.0]),
               dict(vs=[1.0, float("nan")]), dict(ks=[2.0 ** 65, 1.0]), dict(ks=[1.0, 2.0 ** -65])):
        assert make(**kw) == kb.KVP_ERR_INVALID_ARG, kw


def test_null_pools_are_refused():
    kb = ensure_built()
    lib, null, p = kb.lib(), ctypes.c_void_p(), ctypes.c_void_p(256)
    BAD = kb.KVP_ERR_INVALID_ARG
    for name in ("rotary_store_cache_axes", "rotary_store_latent_axes", "rotary_store_fp4"):
        assert getattr(lib, name)(null, 0, p, 8, 8, 1, p, 8, p, 8, p, 1, p, 1, p, p, 2, 8, 0, 1.0, p, 8, 8, null) == BAD
    assert lib.load_cache_fp4(null, 0, p, 1, p, p, null) == BAD
    n = ctypes.c_size_t()
    assert lib.paged_fp4_attention_workspace_size(null, 1, 1, 1, 16, ctypes.byref(n)) == BAD
    assert lib.paged_fp4_attention(null, 0, p, 1, 1, 1, null, p, 1, 1, 0, null, p, 16, 0, 0, 1.0, p, p, 256, null) == BAD


def test_the_pairs_axes():
    kb = ensure_built()
    assert kb.pair_axes((2, 1, 3)) == [0, 0, 1, 2, 2, 2]
    assert kb.pair_axes((2, 1, 3), interleave=True) == [0, 1, 2, 0, 2, 2]
    assert kb.pair_axes((0, 2)) == [1, 1]
    for bad in ((), (1, -1), (1,) * 9):
        with pytest.raises(ValueError):
            kb.pair_axes(bad)
    plan = kb.RotaryPlan(12, device="cpu", sections=(2, 1, 3), interleave=True)
    assert plan.axes == 3 and plan.pair_axis.tolist() == [0, 1, 2, 0, 2, 2] and plan.pair_axis.dtype == torch.uint8
    assert plan.freqs.tolist() == kb.RotaryPlan(12, device="cpu").freqs.tolist()
    one = kb.RotaryPlan(12, device="cpu", sections=(6,))
    assert one.axes == 1 and one.pair_axis is None
    own = kb.RotaryPlan(12, device="cpu", sections=(2, 1, 3), per_axis=True).freqs.tolist()
    assert own == [f for n in (4, 2, 6) for f in kb.RotaryPlan(n, device="cpu").freqs.tolist()]
    for bad in ((2, 1), (4, 4)):
        with pytest.raises(ValueError, match="add up"):
            kb.RotaryPlan(12, device="cpu", sections=bad)


def plan(axes):
    return types.SimpleNamespace(rotary_dim=16, layout=0, attn_factor=1.0, axes=axes, freqs=on(8, torch.int64),
                                 pair_axis=on(8, torch.uint8))


def fp4_pool(kb):
    return types.SimpleNamespace(dtype=kb.KVP_BF16, device_index=0, handle=None, kv_heads=HKV, head_dim=D, page_size=16)


def arguments(kb, call):
    i32, pool = torch.int32, fp4_pool(kb)
    rows = dict(k=on((N, HKV, D)), v=on((N, HKV, D)))
    if call in ("rotary_store_fp4", "rotary_store_cache_axes"):
        t = dict(q=on((N, H, D)), **rows, positions=on((2, N), i32), out_loc=on(N, i32), q_out=on((N, H, D)))
        f = kb.rotary_store_fp4 if call == "rotary_store_fp4" else kb.rotary_store_cache

        def run(x):
            f(pool, 0, x["q"], x["k"], x["v"], x["positions"], x["out_loc"], plan(2), x["q_out"], stream=0)
    elif call == "store_cache_fp4":
        t = dict(**rows, out_loc=on(N, i32))

        def run(x):
            kb.store_cache_fp4(pool, 0, x["k"], x["v"], x["out_loc"], stream=0)
    elif call == "load_cache_fp4":
        t = dict(slots=on(N, i32), k_out=on((N, HKV, D)), v_out=on((N, HKV, D)))

        def run(x):
            kb.load_cache_fp4(pool, 0, x["slots"], x["k_out"], x["v_out"], stream=0)
    else:
        t = dict(q=on((B, C, H, D)), table=on((B, 3), i32), context_lens=on(B, i32), out=on((B, C, H, D)),
                 workspace=on(256, torch.uint8), q_lens=on(B, i32), table_rows=on(B, i32))

        def run(x):
            kb.paged_fp4_attention(pool, 0, x["q"], x["table"], 0, x["context_lens"], 0, 1.0, x["out"], x["workspace"],
                                   q_lens=x["q_lens"], table_rows=x["table_rows"], stream=0)
    return run, t


CALLS = ["rotary_store_fp4", "rotary_store_cache_axes", "store_cache_fp4", "load_cache_fp4", "paged_fp4_attention"]


@pytest.mark.parametrize("call", CALLS)
def test_tensors_elsewhere_are_refused(call, monkeypatch):
    kb = ensure_built()
    library = Library()
    monkeypatch.setattr(kb, "lib", lambda: library)
    run, tensors = arguments(kb, call)
    run(tensors)
    made = ["rotary_store_fp4" if call == "store_cache_fp4" else call]
    assert library.calls == made
    for t in tensors.values():
        for index, error in ((1, ValueError), (None, TypeError)):
            t.index = index
            with pytest.raises(error, match="device|CUDA"):
                run(tensors)
            t.index = 0
    assert library.calls == made


@pytest.mark.parametrize("call", CALLS)
def test_shapes_and_types_are_refused(call, monkeypatch):
    kb = ensure_built()
    library = Library()
    monkeypatch.setattr(kb, "lib", lambda: library)
    run, tensors = arguments(kb, call)
    for name, t in tensors.items():
        if name == "workspace":
            continue
        for bad in (on(t.shape, torch.float16), on((*t.shape[:-1], t.shape[-1] + 1), t.dtype)):
            if name == "table" and bad.dtype == t.dtype:
                continue  # another width is another table
            with pytest.raises((TypeError, ValueError)):
                run({**tensors, name: bad})
    assert library.calls == []


def test_positions_of_a_plan(monkeypatch):
    kb = ensure_built()
    library = Library()
    monkeypatch.setattr(kb, "lib", lambda: library)
    run, t = arguments(kb, "rotary_store_fp4")
    for bad in (on((3, N), torch.int32), on(N, torch.int32), on((N, 2), torch.int32).T.as_subclass(On),
                on((1, N), torch.int32).expand(2, N).as_subclass(On)):
        with pytest.raises(ValueError, match="positions"):
            run({**t, "positions": bad})
    run({**t, "positions": on((2, 2 * N), torch.int32)[:, :N].as_subclass(On)})  # rows that lie apart
    pool = fp4_pool(kb)
    with pytest.raises(ValueError, match="plan"):
        kb.rotary_store_fp4(pool, 0, t["q"], t["k"], t["v"], t["positions"], t["out_loc"], None, t["q_out"], stream=0)
    with pytest.raises(ValueError):
        kb.store_cache_fp4(pool, 0, None, None, t["out_loc"], stream=0)
    assert library.calls == ["rotary_store_fp4"]


def test_four_bit_buffers_of_other_shapes():
    kb = ensure_built()
    codes, scales = on((1, 4, 16, 2, 2, 32), torch.uint8), on((1, 4, 2, 16, 2, 4), torch.uint8)
    for c, s, e in ((on((1, 4, 16, 2, 2, 32), torch.int8), scales, TypeError), (codes[0].as_subclass(On), scales, ValueError),
                    (codes, on((1, 3, 2, 16, 2, 4), torch.uint8), ValueError), (codes, on(scales.shape, torch.int8), TypeError)):
        with pytest.raises(e):
            kb.Fp4Pool(c, s, kb.KVP_BF16)
    with pytest.raises(ValueError):
        kb.Fp4Pool(codes, scales, 7)
    for g in ([1.0, 1.0], []):
        with pytest.raises(ValueError, match="one a layer"):
            kb.Fp4Pool(codes, scales, kb.KVP_BF16, k_scale=g, error_word=on(1, torch.int32))
