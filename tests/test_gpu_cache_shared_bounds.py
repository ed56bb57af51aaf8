"""Shared attention whose groups are malformed, between guards; and calls that share nothing, of many rows."""
import math

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

from .test_gpu_cache_shared import BF16, F32, KINDS, Case, both, ints

pytestmark = pytest.mark.gpu

LEAST, MOST = -2 ** 31, 2 ** 31 - 1


def guarded(case):
    """The call with each buffer that it writes between bytes that it must leave alone."""
    B, T_q, hq, d = case.q.shape
    need = kda.cache_attention_shared_workspace_size(B, T_q, hq, case.pool.k.shape[1], d, case.page, case.table.shape[1],
                                                     case.prefix_table.shape[1], case.prefix_table.shape[0])
    ws = torch.full((need + (2 << 12),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((B + 2, T_q, hq, d), 7.0, dtype=case.q.dtype, device="cuda")
    lse = torch.full((B + 2, T_q, hq), 7.0, device="cuda")
    case.run(out=out[1: B + 1], lse=lse[1: B + 1], workspace=ws[1 << 12: need + (1 << 12)])
    assert bool((ws[: 1 << 12] == 0xA5).all()) and bool((ws[need + (1 << 12):] == 0xA5).all())
    assert bool((out[:: B + 1] == 7).all()) and bool((lse[:: B + 1] == 7).all())
    return out[1: B + 1], lse[1: B + 1]


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("T_q, hq, hk, d, many", [(1, 4, 2, 64, 1), (3, 16, 2, 128, 1), (1, 8, 1, 96, 9)])
def test_malformed_groups_write_what_is_theirs(dtype, T_q, hq, hk, d, many):
    case = Case(12, T_q, hq, hk, d, 16, dtype, [(64, [T_q + 4, 60, 7] * many), (48, [7, 8] * many)])
    n = 5 * many
    inputs = [case.pool.k, case.pool.v, case.pool.k_scale, case.pool.v_scale, case.q, case.table, case.prefix_table, case.lengths]
    before = [t.clone() for t in inputs]
    for cu in ([0, n, 0], [-5, 3, 99], [n - 1, 2, 1], [MOST, LEAST, n], [LEAST, MOST, LEAST], [0, MOST, MOST], [n, 0, n]):
        case.cu.copy_(ints(cu))
        guarded(case)
    for cu in ([0, 0, 0], [n, n, n]):                      # nothing shared: each over its own row
        case.cu.copy_(ints(cu))
        case.check(*guarded(case))
    case.cu.copy_(ints([0, 3 * many, n]))
    for shared in ([MOST, LEAST], [LEAST, MOST], [-1, 0]):   # clamped: prefixes that none sees all of, or none
        case.shared.copy_(ints(shared))
        case.check(*guarded(case))
    for a, b in zip(inputs, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T_q, hq, hk, d", [(9, 4, 2, 128), (20, 4, 2, 80), (65, 2, 2, 112), (17, 1, 1, 64), (3, 24, 2, 96)])
@pytest.mark.parametrize("longest", [200, 1024, 1025, 3001])
def test_nothing_shared_by_many_rows(dtype, T_q, hq, hk, d, longest):
    """More rows a head than 16, whose kernel goes by the block table's room: cache_attention, but for roundings."""
    own = [longest, T_q, 0, longest // 2, T_q - 1, longest - 1, 3]
    case = Case(31, T_q, hq, hk, d, 32, dtype, [], before=own)
    o, lse = both(case)
    want, want_lse = kda.cache_attention(case.q, case.pool, case.table, case.lengths, return_lse=True)
    case.check(want, want_lse)
    assert torch.equal(lse == -math.inf, want_lse == -math.inf)
    again = Case(31, T_q, hq, hk, d, 32, dtype, [(0, [longest, T_q]), (31, [])], before=own[2:])   # groups without a whole page
    both(again)
