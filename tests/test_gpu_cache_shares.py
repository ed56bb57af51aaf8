"""Attention over the cache with items whole and cut: the same tokens under block tables with little and much room, and
under windows that allow few and many steps, each against the 64-bit definition."""
import pytest
import torch

from .test_gpu_cache_ops import BF16, F32, _run_and_check, _setup

pytestmark = pytest.mark.gpu

CASES = [(3, 1, 8, 2, 64, 16, [0, 1, 300]), (2, 4, 4, 2, 128, 64, [700, 33]), (2, 3, 3, 3, 80, 32, [95, 411]),
         (3, 8, 8, 2, 128, 16, [8, 130, 777]), (1, 20, 6, 1, 112, 64, [1500]), (40, 1, 8, 8, 32, 16, [(7 * i) % 50 for i in range(40)]),
         (2, 2, 32, 1, 128, 128, [900, 260])]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]))
@pytest.mark.parametrize("window, sinks", [(0, 0), (100, 5), (2500, 3)])
def test_little_and_much_room(dtype, case, window, sinks):
    q, cache, table, lengths = _setup(21 + window, *case, dtype)
    page = case[5]
    room = torch.full((table.shape[0], 80000 // page - table.shape[1]), -1, dtype=torch.int32, device="cuda")
    far = table[:, :1].expand(-1, 9)                       # held, but beyond every length
    wide = torch.cat([table, far, room], 1).contiguous()
    a, a_lse = _run_and_check(q, cache, table, lengths, window=window, sinks=sinks)
    b, b_lse = _run_and_check(q, cache, wide, lengths, window=window, sinks=sinks)
    again, _ = _run_and_check(q, cache, wide, lengths, window=window, sinks=sinks)
    assert torch.equal(again, b)
    assert torch.equal(torch.isinf(a_lse), torch.isinf(b_lse))


@pytest.mark.parametrize("dtype, T_q", [(BF16, 1), (BF16, 8), (F32, 2)])
def test_one_long_among_short(dtype, T_q):
    lengths = [T_q + i % 5 for i in range(60)] + [3000] + [T_q] * 3
    q, cache, table, lengths = _setup(31, 64, T_q, 8, 2, 128, 64, lengths, dtype)
    _run_and_check(q, cache, table, lengths)
    _run_and_check(q, cache, table, lengths, window=1000, sinks=1)


@pytest.mark.parametrize("dtype, T_q", [(BF16, 1), (BF16, 4), (BF16, 16), (F32, 3)])
def test_every_row_empty_or_one_token(dtype, T_q):
    """Shares of items of a single step, most of them cut nowhere, some rows before the first token."""
    lengths = [i % 3 for i in range(96)]
    q, cache, table, lengths = _setup(33, 96, T_q, 8, 4, 128, 16, lengths, dtype, wide=4)
    room = torch.full((96, 6000), -1, dtype=torch.int32, device="cuda")
    _run_and_check(q, cache, torch.cat([table, room], 1).contiguous(), lengths)
