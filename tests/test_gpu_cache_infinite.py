"""Attention with infinite queries, the same in every kernel: a channel of -inf against keys of one sign makes every score of
its row -inf, which gives 0 and a log-sum of -inf; +inf, both signs, or a zero among the keys give NaN.

Other rows stay what they were but for roundings: rows of a warp move the references of their sums together, so a row that has
none moves them at other tokens.  Each of the two results is within the bound of the attention tests, at these sizes (128
channels, 9,000 tokens, |q k| / sqrt(d) summed up to 24) 2 (2^-24 (2 128 + 8) 24 + 2^-20 + 2^-24 (9000 / 16 + 64)) < 2^-10 for fp32, and
2^-8 + 2 2^-11 more than that for bf16."""
import math

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# fp32; bf16 with few rows a head, and with more than 16 of narrow and of wide heads; whole items and shares
CASES = [(F32, 1, 2, 128, 200), (F32, 5, 4, 64, 5000), (F32, 12, 4, 80, 90), (BF16, 1, 2, 128, 200), (BF16, 4, 4, 64, 5000),
         (BF16, 9, 4, 64, 200), (BF16, 9, 4, 128, 200), (BF16, 12, 4, 96, 9000), (BF16, 70, 1, 128, 300)]


def _other_rows(o, lse, want, want_lse):
    tol = 2.0 ** -9 + (2.0 ** -6 if o.dtype == BF16 else 0.0)
    assert bool(((o.float() - want.float()).abs() <= tol * want.float()).all()) and bool(((lse - want_lse).abs() <= 2.0 ** -9).all())


def _case(T_q, group, d, length, scale=1.0):
    g = torch.Generator().manual_seed(length + d)
    heads, page = 2, 32
    n_pages = -(-length // page)
    codes = torch.randint(0x30, 0x48, (n_pages, heads, page, d), generator=g, dtype=torch.uint8).cuda()   # 0.5 to 4
    ones = torch.full((n_pages, heads), scale, device="cuda")
    cache = kda.PagedCache(codes.view(torch.float8_e4m3fn), codes.clone().view(torch.float8_e4m3fn), ones, torch.ones_like(ones))
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    q = torch.randn(1, T_q, heads * group, d, generator=g).cuda()
    return q, cache, table, torch.full((1,), length, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype, T_q, group, d, length", CASES)
def test_all_scores_minus_infinity(dtype, T_q, group, d, length):
    q, cache, table, lengths = _case(T_q, group, d, length)
    q = q.to(dtype)
    want, want_lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    one = q.clone()
    one[0, T_q // 2, 1, 3] = -math.inf                     # one row
    o, lse = kda.cache_attention(one, cache, table, lengths, return_lse=True)
    mine = torch.zeros(1, T_q, q.shape[2], dtype=torch.bool, device="cuda")
    mine[0, T_q // 2, 1] = True
    assert not bool(o[mine].any()) and bool((lse[mine] == -math.inf).all())
    _other_rows(o[~mine], lse[~mine], want[~mine], want_lse[~mine])
    one[..., d - 1] = -math.inf                            # every row, some with two such channels
    o, lse = kda.cache_attention(one, cache, table, lengths, return_lse=True)
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    # nothing but the infinity and its neighbours of the largest and the smallest size, keys of a tiny scale
    q, cache, table, lengths = _case(T_q, group, d, length, 2.0 ** -60)
    for fill in (0.0, 3e38, -3e38, 1e-38):
        alone = torch.full_like(q, fill).to(dtype)
        alone[..., 5] = -math.inf
        o, lse = kda.cache_attention(alone, cache, table, lengths, return_lse=True)
        assert not bool(o.any()) and bool((lse == -math.inf).all()), fill


@pytest.mark.parametrize("dtype, T_q, group, d, length", CASES)
def test_no_number(dtype, T_q, group, d, length):
    q, cache, table, lengths = _case(T_q, group, d, length)
    q = q.to(dtype)
    want, want_lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    row = torch.zeros(1, T_q, q.shape[2], dtype=torch.bool, device="cuda")
    row[0, T_q // 2, 1] = True
    for values in ({3: math.inf}, {3: math.inf, 4: -math.inf}, {3: math.nan}, {3: math.nan, 4: -math.inf}):
        odd = q.clone()
        for at, v in values.items():
            odd[0, T_q // 2, 1, at] = v
        o, lse = kda.cache_attention(odd, cache, table, lengths, return_lse=True)
        assert bool(torch.isnan(o[row]).all()) and bool(torch.isnan(lse[row]).all()), values
        _other_rows(o[~row], lse[~row], want[~row], want_lse[~row])
    cache.k.view(torch.uint8)[0, :, 7, 3] = 0              # the first page's token 7: minus infinity times zero
    odd = q.clone()
    odd[0, T_q // 2, 1, 3] = -math.inf
    o, lse = kda.cache_attention(odd, cache, table, lengths, return_lse=True)
    assert bool(torch.isnan(o[row]).all()) and bool(torch.isnan(lse[row]).all())
