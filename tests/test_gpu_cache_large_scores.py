"""Attention whose scores are far beyond what differences of 32-bit numbers resolve: one token's score is the largest by more than any
rounding of scores of that size, so its value is the output and its score the log-sum.

Queries are between 1 and 1.13 times one size, keys between 2^-3 and 2^-2, the one token's 0.56: in units of the size times sqrt(d)
its score is 0.56 and more, the others' 0.28 and less.  They are 64 times the size apart times two and more, so all other weights
vanish in 32 bits, and scores are off by 2^-24 (2 d + 8) of themselves.  The one weight need not be 1 itself: it is divided by its own
sum, off by 2^-21 (two fp16 pieces) and two roundings with fp32 queries, by 2^-11 with bf16 ones, which is under half a step of the
output, whose value is a code times a power of two.
"""
import math

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("size", [1.0, 2.0 ** 16, 2.0 ** 24, 2.0 ** 27, 2.0 ** 33, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("dtype, T_q, group, d", [(BF16, 1, 2, 64), (F32, 1, 2, 64), (F32, 7, 4, 128), (BF16, 3, 4, 128), (BF16, 9, 4, 64), (BF16, 9, 4, 128)])
@pytest.mark.parametrize("length, room", [(60, 0), (333, 0), (333, 300), (3000, 0)])
def test_one_token_counts(dtype, T_q, group, d, size, length, room):
    heads, page = 2, 16
    g = torch.Generator().manual_seed(length + d)
    n_pages = -(-length // page)
    best = length - T_q - 5                                # seen by every row
    k = torch.randint(0x20, 0x28, (n_pages, heads, page, d), generator=g, dtype=torch.uint8)     # 2^-3 to 2^-2
    k[best // page, :, best % page] = 0x31
    v = (torch.randn(n_pages, heads, page, d, generator=g) * 40).to(torch.float8_e4m3fn)
    scale = torch.exp2(torch.randint(-6, 7, (n_pages, heads), generator=g).float())              # of v
    cache = kda.PagedCache(k.view(torch.float8_e4m3fn).cuda(), v.cuda(), torch.ones(n_pages, heads, device="cuda"), scale.cuda())
    table = torch.full((1, n_pages + room), -1, dtype=torch.int32)
    table[0, :n_pages] = torch.arange(n_pages)
    q = (torch.rand(1, T_q, heads * group, d, generator=g) * 0.125 + 1.0).to(dtype).float()
    q = (q * size * 64).to(dtype).cuda()
    o, lse = kda.cache_attention(q, cache, table.cuda(), torch.tensor([length], dtype=torch.int32, device="cuda"), return_lse=True)
    score = q.double().sum(-1) * 0.5625 / math.sqrt(d)
    want = (v[best // page, :, best % page].float() * scale[best // page][:, None]).repeat_interleave(group, 0).to(dtype).cuda()
    if dtype == BF16:
        assert torch.equal(o, want.expand_as(o))
    else:
        assert bool(((o - want).abs() <= 2.0 ** -20 * want.abs()).all())
    assert bool(((lse.double() - score).abs() <= 2.0 ** -24 * (2 * d + 16) * score).all())
