"""What bounds a four-bit cache's calls beside a long request: the step's own lengths, and a workspace of limited size."""

import pytest

from test_gpu_fp4_cache import Steps, kb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("host", [None, "prefill_step", "verify_step"])
def test_steps_beside_a_long_request(kb, monkeypatch, host):  # noqa: F811
    s = Steps(kb, "bf16", 32, 8, 128, 16, "block")
    for r in (1, 4, 5):
        s.cache.new(r)
    s.cache.append([5] * 700)
    given, attend = [], kb.paged_fp4_attention
    monkeypatch.setattr(kb, "paged_fp4_attention", lambda *a, **kw: given.append(kw["max_context"]) or attend(*a, **kw))
    s.step([1, 4], 100, host=host)
    s.step([4, 1], 30, host=host)
    s.step([4], 130, host=host)
    assert given == [256, 256, 256, 256, 512, 512]
