"""The binding without its module of C++ marshalling, and with one of another torch: its calls go through ctypes (CPU only)."""

import importlib
import sys
import types
import warnings

import pytest
import torch

from libbuild import ensure_built
from test_operator_devices import on

NAME = "paged_decode_attention_store_gb300._marshal"


def refused_by_the_library(kb):
    """A rotary store that passes the binding's checks; the library refuses its pool."""
    pool = types.SimpleNamespace(dtype=kb.KVP_BF16, device_index=0, handle=None, kv_heads=2, head_dim=64)
    plan = types.SimpleNamespace(rotary_dim=16, layout=0, attn_factor=1.0, freqs=on(8, torch.int64))
    i = on(3, torch.int32)
    with pytest.raises(kb.KvpError) as e:
        kb.rotary_store_cache(pool, 0, None, on((3, 2, 64)), on((3, 2, 64)), i, i, plan, None, stream=0)
    assert e.value.code == kb.KVP_ERR_INVALID_ARG


@pytest.mark.parametrize("module", [None, types.SimpleNamespace(built_for="torch 1.0 Python 3.4"), types.SimpleNamespace()])
def test_a_module_that_is_missing_or_does_not_fit(monkeypatch, module):
    kb = ensure_built()
    package = importlib.import_module("paged_decode_attention_store_gb300")
    monkeypatch.setattr(kb, "_marshal", None)
    monkeypatch.setitem(sys.modules, NAME, module)
    monkeypatch.delattr(package, "_marshal", raising=False)
    if module is not None:
        monkeypatch.setattr(package, "_marshal", module, raising=False)
    with pytest.warns(RuntimeWarning, match="_marshal.so is not used"):
        refused_by_the_library(kb)
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # said once
        assert kb._native() is None
        refused_by_the_library(kb)


def test_the_module_that_was_built():
    kb = ensure_built()
    from paged_decode_attention_store_gb300 import build

    kb._marshal = None
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert kb._native().built_for == build.marshal_for()


def test_another_torch_builds_it_anew(monkeypatch, tmp_path):
    ensure_built()
    from paged_decode_attention_store_gb300 import build

    made = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "MARSHAL_FOR", str(tmp_path / "_build" / "marshal_for"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "_run", lambda cmd: made.append(cmd) or open(cmd[cmd.index("-o") + 1], "w").close())
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    build.build_marshal()
    build.build_marshal()
    assert len(made) == 1
    monkeypatch.setattr(torch, "__version__", "1.0")
    build.build_marshal()
    build.build_marshal()
    assert len(made) == 2 and any("torch 1.0" in x for x in made[1])
