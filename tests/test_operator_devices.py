"""The rotary, latent and expanded calls refuse a tensor of the host's memory or of another device before anything
reaches the library (CPU only: tensors that say they are on a device, and a library that records its calls)."""

import types

import pytest
import torch

from libbuild import ensure_built

B, C, H, D, DC, DR, N = 2, 1, 4, 64, 32, 16, 2


class On(torch.Tensor):
    """A host tensor that says it is on a device: ``index`` (None: the host)."""

    index = 0

    @property
    def is_cuda(self):
        return self.index is not None

    def get_device(self):
        return -1 if self.index is None else self.index


def on(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(On)


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


def arguments(kb, call):
    """(the call, its pool or None, its named tensors)."""
    i32 = torch.int32
    plan = types.SimpleNamespace(rotary_dim=DR, layout=0, attn_factor=1.0)
    if call == "rotary_store_cache":
        pool = types.SimpleNamespace(dtype=kb.KVP_BF16, device_index=0, handle=None, kv_heads=2, head_dim=D)
        t = dict(q=on((N, H, D)), k=on((N, 2, D)), v=on((N, 2, D)), positions=on(N, i32), out_loc=on(N, i32),
                 freqs=on(DR // 2, torch.int64), q_out=on((N, H, D)))

        def run(x):
            plan.freqs = x["freqs"]
            kb.rotary_store_cache(pool, 0, x["q"], x["k"], x["v"], x["positions"], x["out_loc"], plan, x["q_out"], stream=0)
    elif call == "rotary_store_latent":
        pool = types.SimpleNamespace(dtype=kb.KVP_BF16, device_index=0, handle=None, latent_dim=DC, rope_dim=DR)
        t = dict(q_pe=on((N, H, DR)), latent=on((N, DC)), k_pe=on((N, DR)), positions=on(N, i32), out_loc=on(N, i32),
                 freqs=on(DR // 2, torch.int64), q_pe_out=on((N, H, DR)))

        def run(x):
            plan.freqs = x["freqs"]
            kb.rotary_store_latent(pool, 0, x["q_pe"], x["latent"], x["k_pe"], x["positions"], x["out_loc"], plan,
                                   x["q_pe_out"], stream=0)
    elif call == "paged_latent_attention":
        pool = types.SimpleNamespace(dtype=kb.KVP_BF16, device_index=0, handle=None, head_dim=DC + DR, latent_dim=DC)
        t = dict(q=on((B, C, H, DC + DR)), table=on((B, 3), i32), context_lens=on(B, i32), out=on((B, C, H, DC)),
                 workspace=on(256, torch.uint8), q_lens=on(B, i32), table_rows=on(B, i32))

        def run(x):
            kb.paged_latent_attention(pool, 0, x["q"], x["table"], 0, x["context_lens"], 0, 1.0, x["out"], x["workspace"],
                                      q_lens=x["q_lens"], table_rows=x["table_rows"], stream=0)
    else:
        t = dict(q=on((N, H, D + DR)), k=on((N, H, D)), k_pe=on((N, DR)), v=on((N, H, D)), q_start=on(B, i32),
                 k_start=on(B, i32), out=on((N, H, D)), error_word=on(1, i32))

        def run(x):
            kb.latent_prefill_attention(x["q"], x["k"], x["k_pe"], x["v"], x["q_start"], x["k_start"], N, 1.0, x["out"],
                                        error_word=x["error_word"], stream=0)
    return run, t


@pytest.mark.parametrize("call", ["rotary_store_cache", "rotary_store_latent", "paged_latent_attention",
                                  "latent_prefill_attention"])
def test_tensors_elsewhere_are_refused(call, monkeypatch):
    kb = ensure_built()
    library = Library()
    monkeypatch.setattr(kb, "lib", lambda: library)
    run, tensors = arguments(kb, call)
    run(tensors)
    assert library.calls == [call]
    for name, t in tensors.items():
        for index, error in ((1, ValueError), (None, TypeError)):
            if name == "q" and call == "latent_prefill_attention" and index == 1:
                continue  # q names the device there: the others are then elsewhere
            t.index = index
            with pytest.raises(error, match="device|CUDA"):
                run(tensors)
            t.index = 0
    assert library.calls == [call]


def test_the_queries_of_a_prompt_elsewhere(monkeypatch):
    kb = ensure_built()
    library = Library()
    monkeypatch.setattr(kb, "lib", lambda: library)
    run, tensors = arguments(kb, "latent_prefill_attention")
    tensors["q"].index = 1
    with pytest.raises(ValueError, match="device"):
        run(tensors)
    for t in tensors.values():
        t.index = None
    with pytest.raises(TypeError, match="CUDA"):
        run(tensors)
    assert library.calls == []
