"""The compiled marshalling of the global-attention operators, without a GPU: what it does not take it leaves to
the checks in Python, and nothing runs without it."""
import inspect

import pytest
import torch

import gated_delta_rule_34_gb300 as kda
from gated_delta_rule_34_gb300 import build, cache


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_missing_binding_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="build it with"):
        cache._binding.__wrapped__()


# None in the place of every tensor, a tensor on the CPU in the place of one: neither is taken, and neither crashes
@pytest.mark.parametrize("name", ["rotary", "cache_write", "cache_read", "cache_attention"])
def test_odd_arguments_are_left_alone(name):
    entry, public = getattr(cache._binding(), name), getattr(kda, name)
    n = len(inspect.signature(public).parameters)
    assert entry(*[None] * n) is None
    x = torch.zeros(1, 2, 4, 64)
    for i in range(n):
        assert entry(*[x if j == i else None for j in range(n)]) is None
    assert entry(*[x] * n) is None
    assert entry(*[(x, x, x, x)] * n) is None
    with pytest.raises(TypeError, match="arguments"):
        entry(*[None] * (n + 1))


def test_public_calls_name_what_is_wrong():
    x = torch.zeros(1, 2, 4, 64)
    pool = kda.cache_new(2, 4, 16, 64, device="cpu")
    i = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: kda.rotary(x, x, i[0], torch.zeros(32, dtype=torch.float64)),
                 lambda: kda.cache_write(pool, x, x, i, i[0]),
                 lambda: kda.cache_read(pool, i, i[0], 1),
                 lambda: kda.cache_attention(x, pool, i, i[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
