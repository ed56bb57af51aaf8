"""The many-row attention's bounded waits, run out: loaders that load only some tiles, or products that stop after some
tiles, with a limit of 3 ms.  The call returns, its outputs are NaN, and the context goes on to give the right ones.  No fault:
every wait of the kernel ends by itself."""
import time

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

from .test_gpu_cache_ops import BF16, _setup

pytestmark = pytest.mark.gpu

ALL = 1 << 24


@pytest.fixture(autouse=True)
def off():
    yield
    kda.selftest_attention_stall()


# 700 and 1000 tokens are 6 and 8 tiles, one CTA's with 32 items; 100,000 are 782, shared out, ten tiles and more in every share
@pytest.mark.parametrize("lengths", [[700, 1000] * 8, [100_000, 99_900]])
@pytest.mark.parametrize("loads, tiles", [(0, ALL), (1, ALL), (2, ALL), (3, ALL), (4, ALL), (5, ALL), (ALL, 0), (ALL, 1), (ALL, 3), (ALL, 4)])
def test_waits_run_out(lengths, loads, tiles):
    q, cache, table, lengths = _setup(41, len(lengths), 8, 8, 2, 128, 64, lengths, BF16)
    want, want_lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    assert bool(torch.isfinite(want).all())
    torch.cuda.synchronize()
    kda.selftest_attention_stall(loads, tiles, 3000)
    t0 = time.perf_counter()
    o, lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 20.0
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
    kda.selftest_attention_stall()
    o, lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_enough_is_enough():
    """Stopping after all that a CTA has to do, or where no such kernel runs, changes nothing."""
    q, cache, table, lengths = _setup(42, 16, 8, 8, 2, 128, 64, [700, 1000] * 8, BF16)
    few, want_few = q[:, :4].contiguous(), kda.cache_attention(q[:, :4].contiguous(), cache, table, lengths)
    want = kda.cache_attention(q, cache, table, lengths)
    kda.selftest_attention_stall(8, 8, 1_000_000)
    assert torch.equal(kda.cache_attention(q, cache, table, lengths), want)
    kda.selftest_attention_stall(0, 0, 3000)
    assert torch.equal(kda.cache_attention(few, cache, table, lengths), want_few)


def test_the_long_item_alone():
    """A tile does for 100 tokens and not for 600."""
    q, cache, table, lengths = _setup(43, 4, 8, 4, 1, 128, 64, [600, 100, 100, 100], BF16)
    want = kda.cache_attention(q, cache, table, lengths)
    kda.selftest_attention_stall(1, ALL, 3000)
    o = kda.cache_attention(q, cache, table, lengths)
    assert bool(torch.isnan(o[0]).all()) and torch.equal(o[1:], want[1:])
