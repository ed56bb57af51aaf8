"""Attention with the work shared out over many (sequence, row tile) pairs: more than one a thread where each CTA looks for its
share, as many as are shared out at all and one more, and prompts of many row tiles.  Each against the 64-bit definition."""
import pytest
import torch

import gated_delta_rule_34_gb300 as kda

from .test_gpu_cache_ops import BF16, F32, _check_attention, _run_and_check, _setup

pytestmark = pytest.mark.gpu


def _with_room(case, dtype, pages=200):
    """The block table gets room for 3,200 tokens and more, so that items are cut."""
    q, cache, table, lengths = _setup(sum(case[6]) + case[0], *case, dtype)
    room = torch.full((case[0], pages), -1, dtype=torch.int32, device="cuda")
    return q, cache, torch.cat([table, room], 1).contiguous(), lengths


# a thread of the few-row kernel has 2 and more pairs from 129 sequences on
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B", [127, 128, 129, 256, 257, 300, 1025])
def test_many_sequences(dtype, B):
    lengths = [(i * 37) % 61 for i in range(B)]
    lengths[B // 3] = 900
    _run_and_check(*_with_room((B, 1, 4, 2, 32, 16, lengths), dtype))


# one of the many-row kernel from 385 on
@pytest.mark.parametrize("B, T_q", [(383, 5), (385, 5), (800, 9)])
def test_many_sequences_of_many_rows(B, T_q):
    lengths = [(i * 29) % 45 for i in range(B)]
    lengths[B // 2] = 700
    _run_and_check(*_with_room((B, T_q, 4, 1, 80, 16, lengths), BF16))


@pytest.mark.parametrize("dtype, d", [(BF16, 32), (BF16, 80), (F32, 64)])
def test_prompts_of_many_row_tiles(dtype, d):
    """The 1,000 newest tokens of 1,000 and of 1,333, 4 rows each: 63 or 125 row tiles a sequence, the first of which see little."""
    _run_and_check(*_with_room((2, 1000, 4, 1, d, 16, [1000, 1333]), dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B", [8191, 8192, 8193])
def test_most_pairs(dtype, B):
    """Up to 8,192 pairs are shared out, beyond that each item is one CTA's, however long."""
    lengths = [i % 3 for i in range(B)]
    lengths[B // 2], lengths[-1] = 48, 40
    _run_and_check(*_with_room((B, 1, 1, 1, 16, 16, lengths), dtype))


def test_most_pairs_of_one_prompt():
    """Row tiles count as well: 2,048 sequences of four tiles are shared out, 2,049 are not."""
    for B in (2048, 2049):
        lengths = [1 + i % 2 for i in range(B)]
        lengths[7] = 45
        q, cache, table, lengths = _with_room((B, 2, 64, 1, 80, 16, lengths), BF16)
        sub = torch.tensor(list(range(0, B, 400)) + [7, B - 1], device="cuda")
        o, lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
        _check_attention(q[sub], cache, table[sub], lengths[sub], o[sub], lse[sub])
        assert bool(torch.isfinite(o).all())
