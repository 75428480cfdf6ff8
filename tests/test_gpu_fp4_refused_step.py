"""A step of a four-bit cache that is refused leaves its queries as they were; the check in C++ and Python's agree."""

import pytest
import torch

from test_gpu_fp4_cache import Steps, kb  # noqa: F401

pytestmark = pytest.mark.gpu


class Counted:
    def __init__(self, native):
        self.native, self.answers = native, []

    def __getattr__(self, name):
        def call(*a):
            code = getattr(self.native, name)(*a)
            if name == "step":
                self.answers.append(code)
            return code
        return call


def test_a_refused_step_turns_no_queries(kb, monkeypatch):  # noqa: F811
    s = Steps(kb, "bf16", 8, 2, 128, 16, "block")
    native = Counted(kb._native())
    monkeypatch.setattr(kb, "_native", lambda: native)
    s.cache.new(0)
    s.step([0], 20)
    assert native.answers == [True]
    q, o, k = ([s.rnd(*n) for _ in range(2)] for n in ((1, 3, 8, 128), (1, 3, 8, 128), (3, 2, 128)))
    wide = s.rnd(3, 5, 128)
    given = [x.clone() for x in q]
    odd = s.rnd(3 * 8 * 128 + 1)[1:].view(1, 3, 8, 128)
    for bad in (dict(q=[q[0], q[1].float()]), dict(q=[q[0], odd]), dict(q=q[:1]), dict(out=[o[0], o[1][:, :2]]),
                dict(out=[o[0], o[1].cpu()]), dict(k=[k[0], k[1][:2]]), dict(v=[k[0], wide[:, 1:4]]), dict(v=[k[0], None]),
                dict(scale=float("nan")), dict(window=5, sinks=5)):
        a = dict(q=q, k=k, v=k, out=o, window=0, scale=1.0, sinks=0)
        a.update(bad)
        with pytest.raises((ValueError, TypeError, IndexError)):
            s.cache.step([0], a["q"], a["k"], a["v"], s.plan, a["out"], a["window"], a["scale"], sinks=a["sinks"])
        assert all(torch.equal(x, y) for x, y in zip(q, given)) and s.cache.lengths[0] == 20
    assert native.answers == [True] + [None] * 8
    s.cache.step([0], tuple(q), tuple(k), [wide[:, 1:3], wide[:, 3:]], s.plan, o, 0, 1.0)  # rows of one projection's output
    assert native.answers[-1] is True and not torch.equal(q[0], given[0]) and s.cache.lengths[0] == 23
    s.cache.check()
