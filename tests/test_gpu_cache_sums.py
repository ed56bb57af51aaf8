"""Attention's sums of values of one sign over long sequences: additions that cut off instead of rounding err one way, and
that grows with the length.

Queries of zeros give every token the weight 1, exactly, and codes are exact in the products, so an output is off by
its sums alone.  The codes span 2^-9 to 448 and their sums pass 2^23, far more bits than 32-bit numbers hold.  Many
sequences share the pages, so that a CTA has whole items and its warps long runs of tokens.

The bound, relative to the output.  A warp adds a step of 16 tokens to its sums at most length / 16 = n times, each addition
rounded: half a step 2^-24 of the sum so far, independent of each other.  Of errors evenly spread over it the
deviation is 2^-24 / sqrt(3) sqrt(n / 3) (the sums grow evenly): six of them are 2^-23 sqrt(n).  The product of a step is cut
off, at most 2^-21 of it; the factors at the end add 2^-21.  More than 16 bf16 rows of more than 64 channels are summed in the
products for 64 tiles of four products, cut off by at most a step 2^-23 of what is summed so far, half of that over the run: 256
2^-24.  An output must be what a number within the bound rounds to.
"""
import math

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype, T_q, group, d", [
    (F32, 1, 4, 128), (F32, 4, 4, 128), (F32, 8, 4, 128), (F32, 16, 4, 128), (F32, 1, 4, 64), (F32, 16, 4, 64),
    (BF16, 1, 4, 128), (BF16, 4, 4, 128), (BF16, 2, 4, 64), (BF16, 4, 4, 64), (BF16, 8, 4, 64), (BF16, 16, 4, 64),
    (BF16, 8, 4, 128), (BF16, 8, 4, 80),
])
@pytest.mark.parametrize("length, B", [(1 << 17, 64), (100_003, 3)])
def test_values_of_one_sign(dtype, T_q, group, d, length, B):
    heads, page = 8, 128
    g = torch.Generator().manual_seed(length + d)
    n_pages = -(-length // page)
    codes = torch.randint(1, 0x7F, (n_pages, heads, page, d), generator=g, dtype=torch.uint8).cuda()
    ones = torch.ones(n_pages, heads, device="cuda")
    cache = kda.PagedCache(codes.view(torch.float8_e4m3fn), codes.view(torch.float8_e4m3fn), ones, ones)
    table = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    q = torch.zeros(B, T_q, heads * group, d, dtype=dtype, device="cuda")
    o, lse = kda.cache_attention(q, cache, table.expand(B, -1).contiguous(), torch.full((B,), length, dtype=torch.int32, device="cuda"),
                                 return_lse=True)
    rows = codes[table.long()].view(torch.float8_e4m3fn).double().transpose(1, 2).flatten(0, 1)
    last = rows[length - T_q: length]                      # tokens that some of the queries do not see
    total = rows[:length].sum(0)
    n = length / 16
    bound = 2.0 ** -23 * math.sqrt(n) + 2.0 ** -20 + (256 * 2.0 ** -24 if dtype == BF16 and d > 64 and T_q * group > 16 else 0.0)
    for i in range(T_q):
        want = ((total - last[i + 1:].sum(0)) / (length - T_q + 1 + i))[None, :, None, :]
        low, high = ((want * (1 + s * bound)).float().to(dtype).float() for s in (-1, 1))
        got = o[:, i].float().view(B, heads, group, d)
        assert bool(((got >= low) & (got <= high)).all()), float(((got.double() - want) / want).abs().max() / bound)
    counts = torch.arange(length - T_q + 1, length + 1, dtype=torch.float64, device="cuda")[None, :, None]
    assert float((lse.double() - counts.log()).abs().max()) <= 2.0 ** -20
