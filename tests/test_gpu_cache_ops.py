"""The global-attention operators on the GPU against plain 64-bit forms.

Tolerances.  Codes and scales are decided by exact arithmetic, so writes and reads must agree bit
for bit.  Rotary: one rounding to the type (half a step, 2^-8 of the value for bf16, 2^-24 for fp32)
plus the 32-bit arithmetic, at most 2^-20 of the pair's length.  Attention: see _check_attention.
"""
import math

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

from . import cache_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _bits(x):
    return x.contiguous().view(torch.uint8).cpu()


# ---------------------------------------------------------------- rotary

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n, hq, hk, d, rot", [
    (1, 16, 4, 128, 128), (1, 1, 1, 16, 2), (7, 5, 5, 64, 64), (3, 3, 1, 80, 16), (33, 8, 2, 96, 50), (2, 64, 8, 256, 250),
    (700, 4, 2, 128, 64), (5, 40, 8, 128, 126), (2, 600, 0, 32, 18), (1300, 2, 1, 64, 32),
])
def test_rotary(dtype, layout, n, hq, hk, d, rot):
    g = _gen(n * 1000 + d + rot)
    q, k = _randn(g, n, hq, d, dtype=dtype), _randn(g, n, hk, d, dtype=dtype) if hk else None
    positions = torch.randint(-(2 ** 31), 2 ** 31 - 1, (n,), generator=g, dtype=torch.int64)
    positions[: n // 2] %= 4096
    positions = positions.to(torch.int32)
    freq = kda.rotary_frequencies(rot, device="cpu")
    got = kda.rotary(q, k, positions.cuda(), freq.cuda(), layout=layout, amplitude=1.25)
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        want = ref.rotary(x.cpu(), positions, freq, layout, 1.25)
        # the angle: 2^31 * 2^-53 rounding of the 64-bit reference and of the operator, plus 32-bit steps
        length = 1.25 * x.cpu().double().abs().amax() * math.sqrt(2)
        err = (y.cpu().double() - want).abs()
        assert bool((err <= HALF_STEP[dtype] * want.abs() + length * 2.0 ** -19).all()), float(err.max())
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout, rot", [("half", 64), ("interleaved", 64), ("half", 50), ("interleaved", 34)])
def test_rotary_strides_batches_and_in_place(layout, rot):
    g = _gen(rot)
    B, T, hq, hk, d = 2, 9, 6, 2, 64
    qkv = _randn(g, B, T, (hq + 2 * hk) * d, dtype=BF16)
    q, k = (qkv[..., a * d: b * d].unflatten(-1, (b - a, d)) for a, b in ((0, hq), (hq, hq + hk)))
    positions = torch.arange(B * T, dtype=torch.int32, device="cuda").view(B, T)
    freq = kda.rotary_frequencies(rot)
    want = kda.rotary(q.contiguous(), k.contiguous(), positions, freq, layout=layout)
    got = kda.rotary(q, k, positions, freq, layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    values = qkv[..., (hq + hk) * d:].clone()
    kda.rotary(q, k, positions, freq, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[..., (hq + hk) * d:], values)


def test_rotary_turns_back():
    g = _gen(3)
    q = _randn(g, 50, 4, 64)
    positions = torch.randint(0, 2 ** 20, (50,), generator=g, dtype=torch.int32).cuda()
    freq = kda.rotary_frequencies(64)
    there, _ = kda.rotary(q, None, positions, freq)
    back, _ = kda.rotary(there, None, -positions, freq)
    # two turns, each off by at most 2^-20 of the pair's length and a rounding
    assert float((back - q).abs().max()) <= float(q.abs().max()) * math.sqrt(2) * 2.0 ** -18


# ---------------------------------------------------------------- writing and reading

def _table(g, B, wide, n_pages):
    return torch.randperm(n_pages, generator=g)[: B * wide].to(torch.int32).view(B, wide)


def _same_cache(cache, want):
    for name in "kv":
        assert torch.equal(getattr(cache, name + "_scale").cpu().double(), want.scale[name])
        got = getattr(cache, name).cpu().float().double()
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want.codes[name], nan=1e9))


def _filled(g, n_pages, heads, page, d):
    """A pool whose codes are any bytes, NaN included, under valid scales."""
    cache = kda.cache_new(n_pages, heads, page, d)
    for name in "kv":
        codes = torch.randint(0, 256, (n_pages, heads, page, d), generator=g, dtype=torch.uint8)
        getattr(cache, name).view(torch.uint8).copy_(codes)
        e = torch.randint(-12, 6, (n_pages, heads), generator=g).float()
        getattr(cache, name + "_scale").copy_(torch.exp2(e))
    return cache


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B, T, heads, d, page, starts", [
    (1, 1, 1, 16, 16, [0]), (3, 1, 2, 128, 64, [0, 5, 63]), (2, 5, 3, 80, 16, [14, 0]), (2, 200, 2, 64, 32, [31, 7]),
    (1, 300, 1, 128, 256, [250]), (2, 130, 2, 128, 128, [127, 128]), (2, 70, 5, 112, 64, [1, 100]),
])
def test_write_fixed(dtype, B, T, heads, d, page, starts):
    g = _gen(B * 100 + T + d)
    wide = (max(starts) + T + page - 1) // page
    n_pages = B * wide + 2
    cache, table = _filled(g, n_pages, heads, page, d), _table(g, B, wide, n_pages)
    want = ref.Cache(cache)
    x = {n: _randn(g, B, T, heads, d) * torch.exp2(torch.randint(-6, 7, (B, T, heads, 1), generator=g).float()).cuda()
         for n in "kv"}
    x = {n: t.to(dtype) for n, t in x.items()}
    kda.cache_write(cache, x["k"], x["v"], table.cuda(), _int32(starts))
    for name in "kv":
        for b in range(B):
            want.write(name, x[name][b], table, b, starts[b])
    _same_cache(cache, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens, starts, page", [
    ([1, 0, 33, 100, 0, 2], [0, 5, 20, 15, 0, 16], 16), ([0, 0, 3], [1, 2, 3], 64), ([1] * 40, list(range(40)), 32),
    ([500, 1], [63, 64], 64),
])
def test_write_packed_and_read_back(dtype, lens, starts, page):
    g = _gen(sum(lens) + page)
    heads, d, B, total = 2, 48, len(lens), sum(lens)
    wide = max((s + n + page - 1) // page for s, n in zip(starts, lens)) + 1
    n_pages = B * wide
    cache, table = _filled(g, n_pages, heads, page, d), _table(g, B, wide, n_pages)
    want = ref.Cache(cache)
    cu = [sum(lens[:i]) for i in range(B + 1)]
    kv = _randn(g, 1, total, 2 * heads * d, dtype=dtype)                # views of one projection
    k, v = (kv[..., i * heads * d: (i + 1) * heads * d].unflatten(-1, (heads, d)) for i in (0, 1))
    kda.cache_write(cache, k, v, table.cuda(), _int32(starts), cu_seqlens=_int32(cu))
    for name, x in (("k", k), ("v", v)):
        for b in range(B):
            want.write(name, x[0, cu[b]: cu[b + 1]], table, b, starts[b])
    _same_cache(cache, want)
    for out in (BF16, F32):
        got = kda.cache_read(cache, table.cuda(), _int32(starts), total, cu_seqlens=_int32(cu), dtype=out)
        for name, y in zip("kv", got):
            rows = [want.values(name, table, b, starts[b] + t) for b in range(B) for t in range(lens[b])]
            assert torch.equal(y[0].cpu(), torch.stack(rows).to(out))


def test_appending_token_by_token_is_one_write():
    """Scales only grow by powers of two, so values that stay in the normal range end up the same."""
    g = _gen(5)
    page, heads, d, T = 16, 2, 32, 40
    table = _table(g, 1, 3, 3)
    x = (torch.randint(8, 16, (1, T, heads, d), generator=g) * torch.exp2(torch.arange(T) % 5)[None, :, None, None]).cuda()
    whole, steps = kda.cache_new(3, heads, page, d), kda.cache_new(3, heads, page, d)
    x = x.to(BF16)
    kda.cache_write(whole, x, -x, table.cuda(), _int32([0]))
    for t in range(T):
        kda.cache_write(steps, x[:, t: t + 1], -x[:, t: t + 1], table.cuda(), _int32([t]))
    for a, b in zip(whole, steps):
        used = [table[0, i] for i in range(3)]
        for i, p in enumerate(used):
            n = min(page, T - i * page)
            assert torch.equal(_bits(a[p, :, :n] if a.dim() == 4 else a[p]), _bits(b[p, :, :n] if b.dim() == 4 else b[p]))
    assert torch.equal(kda.cache_read(whole, table.cuda(), _int32([0]), T, dtype=BF16)[0], x)   # 4 bits fit exactly


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_extremes(dtype):
    """Infinities, NaN, zeros of both signs, the smallest and largest values, all in one page or alone."""
    big, tiny = float(torch.finfo(dtype).max), float(torch.finfo(dtype).tiny)
    rows = [[0.0, -0.0], [math.inf, 3.0], [-math.inf, math.nan], [math.nan, math.nan], [big, -big], [tiny, -tiny],
            [tiny * 2.0 ** -4, 0.0], [448.0, 449.0], [1.75, 1.7578125], [2.0 ** -100, 2.0 ** -93], [big, 1.0]]
    d, page = 16, 16
    x = torch.zeros(len(rows), 1, 1, d)
    for i, r in enumerate(rows):
        x[i, 0, 0, :2] = torch.tensor(r)
    x = x.to(dtype).cuda()
    cache, table = kda.cache_new(len(rows), 1, page, d), torch.arange(len(rows), dtype=torch.int32).view(-1, 1)
    want = ref.Cache(cache)
    kda.cache_write(cache, x, x.flip(-1), table.cuda(), _int32([0] * len(rows)))
    for name, y in (("k", x), ("v", x.flip(-1))):
        for b in range(len(rows)):
            want.write(name, y[b], table, b, 0)
    _same_cache(cache, want)
    assert torch.equal(torch.signbit(cache.k[0, 0, 0, :2].float()).cpu(), torch.tensor([False, True]))


def test_pages_that_are_not_held():
    g = _gen(9)
    heads, d, page = 2, 32, 16
    cache = _filled(g, 6, heads, page, d)
    before = [_bits(t) for t in cache]
    table = _int32([[-1, 6, 2 ** 31 - 1], [-(2 ** 31), 3, -7]])
    x = _randn(g, 2, 48, heads, d, dtype=BF16)
    kda.cache_write(cache, x, x, table, _int32([0, 0]))
    for i, (a, b) in enumerate(zip(before, cache)):
        changed = (a != _bits(b)).view(6, -1).any(1)
        assert not bool(changed[[0, 1, 2, 4, 5]].any())
    k, v = kda.cache_read(cache, table, _int32([0, 0]), 70, dtype=BF16)   # past the table too
    assert int(torch.count_nonzero(k[0])) == 0 and int(torch.count_nonzero(v[0])) == 0
    assert int(torch.count_nonzero(k[1, :16])) == 0 and int(torch.count_nonzero(k[1, 32:])) == 0
    assert int(torch.count_nonzero(k[1, 16:32])) > 0


# ---------------------------------------------------------------- attention

def _check_attention(q, cache, table, lengths, got_o, got_lse, scale=None, window=0, sinks=0):
    """The bound.  A score is a sum of d products: 2^-24 (d + 8) of the sum S of their sizes, with its
    scalings; its exponential adds 2^-21.  Weights go to the product with the values in fp16 (half a step
    2^-11) for bf16 outputs, in two fp16 pieces (2^-21) for fp32 ones; sums of n terms in 32 bits add
    2^-24 (n / 16 + 64).  All of it counts on sum w |v|, twice for the division by the sum; then
    half a step of the output's type.  The half step of an fp16 weight is relative only down to fp16's least
    normal number; below, it is half of 2^-24, with the largest weight (times its page's scale) at 2^12: an error of
    2^-37 of the largest for each token.  With more than 16 bf16 rows a head of more than 64 channels the weights are
    four e5m2 pieces of such an fp16 value with the reference at 2^8: the last one's spacing is 2^-16 4^-3 = 2^-22 there,
    half of it 2^-31 of the reference.
    fp16 queries hold their row's largest value to 2^-25, an error of the score of d 2^-25 S at most."""
    table, lengths = table.cpu(), lengths.cpu()
    d = q.shape[-1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    c = ref.Cache(cache)
    o, lse, weight, size, floor = ref.attention(q, c, table, lengths, scale, window, sinks)
    n = int(lengths.max())
    score = 2.0 ** -24 * (2 * d + 8) * size
    many = q.dtype == BF16 and d > 64 and q.shape[1] * (q.shape[2] // cache.k.shape[1]) > 16
    step = (2.0 ** -11 if q.dtype == BF16 else 2.0 ** -21) + 2.0 ** -21 + 2.0 ** -24 * (n / 16 + 64)
    tol = HALF_STEP[q.dtype] * o.abs() + 2 * (score + step)[..., None] * weight + (2.0 ** -31 if many else 2.0 ** -37) * floor + 1e-30
    err = (got_o.cpu().double() - o).abs()
    finite = torch.isfinite(o)
    assert torch.equal(torch.isnan(got_o.cpu()), torch.isnan(o))
    assert bool((err <= tol)[finite].all()), float((err / tol)[finite].max())
    seen = torch.isfinite(lse)
    assert torch.equal(got_lse.cpu()[~seen & ~torch.isnan(lse)].double(), lse[~seen & ~torch.isnan(lse)])
    lse_tol = score + 2.0 ** -20 + 2.0 ** -22 * lse.abs() + 2.0 ** -24 * (n / 16 + 64)
    assert bool(((got_lse.cpu().double() - lse).abs() <= lse_tol)[seen].all())
    assert not bool(got_o.cpu()[lse == -math.inf].any())


def _setup(seed, B, T_q, hq, hk, d, page, lengths, dtype, spread=3, wide=None, stale=True):
    g = _gen(seed)
    wide = wide or max(1, max((n + page - 1) // page for n in lengths))
    n_pages = B * wide + 1
    cache, table = kda.cache_new(n_pages, hk, page, d), _table(g, B, wide, n_pages)
    if stale:                                    # what no token was written to is not a number
        cache.k.view(torch.uint8).fill_(0x7F)
        cache.v.view(torch.uint8).fill_(0xFF)
    T = max(lengths)
    if T:
        size = torch.exp2(torch.randint(-spread, spread + 1, (B, T, hk, 1), generator=g).float())
        k, v = ((torch.randn(B, T, hk, d, generator=g) * size).cuda() for _ in range(2))
        cu = _int32([sum(lengths[:i]) for i in range(B + 1)])
        pack = [torch.cat([x[b, : lengths[b]] for b in range(B)])[None].contiguous() for x in (k, v)]
        kda.cache_write(cache, pack[0], pack[1], table.cuda(), _int32([0] * B), cu_seqlens=cu)
    q = torch.randn(B, T_q, hq, d, generator=g).to(dtype).cuda()
    return q, cache, table.cuda(), _int32(lengths)


def _run_and_check(q, cache, table, lengths, **kw):
    o, lse = kda.cache_attention(q, cache, table, lengths, return_lse=True, **kw)
    _check_attention(q, cache, table, lengths, o, lse, **kw)
    return o, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B, T_q, hq, hk, d, page, lengths", [
    (1, 1, 1, 1, 16, 16, [1]), (1, 1, 8, 2, 64, 16, [77]), (3, 1, 4, 4, 128, 64, [0, 1, 200]),
    (2, 1, 6, 2, 80, 32, [15, 16]), (2, 1, 7, 1, 96, 16, [17, 129]), (4, 3, 8, 2, 112, 16, [0, 1, 2, 90]),
    (1, 5, 12, 4, 32, 128, [300]), (2, 16, 8, 1, 128, 64, [16, 150]), (1, 1, 16, 1, 48, 256, [513]),
    (1, 7, 20, 4, 128, 32, [1000]), (2, 40, 4, 2, 64, 16, [40, 75]), (1, 1, 40, 1, 128, 64, [65]),
    (1, 1, 130, 1, 64, 32, [99]), (5, 2, 2, 1, 64, 16, [31, 32, 33, 47, 48]),
])
def test_attention(dtype, B, T_q, hq, hk, d, page, lengths):
    _run_and_check(*_setup(sum(lengths) + d + hq, B, T_q, hq, hk, d, page, lengths, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (50, 0), (100, 17), (1000, 3), (64, 300), (33, 16)])
def test_attention_window(dtype, window, sinks):
    _run_and_check(*_setup(window + sinks, 3, 4, 4, 2, 64, 16, [3, 130, 259], dtype), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_many_sequences(dtype):
    lengths = [(i * 37) % 90 for i in range(70)]
    _run_and_check(*_setup(4, 70, 1, 6, 3, 32, 16, lengths, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T_q", [1, 4])
def test_attention_long(dtype, T_q):
    """Long enough to be split many times over."""
    q, cache, table, lengths = _setup(6, 2, T_q, 4, 1, 64, 64, [9001, 4096], dtype)
    _run_and_check(q, cache, table, lengths)
    _run_and_check(q, cache, table, lengths, window=5000, sinks=5)


def test_attention_short_lengths_in_a_wide_table():
    """Room for long sequences, few tokens in them; lengths beyond the table and below zero."""
    q, cache, table, _ = _setup(8, 4, 2, 4, 2, 64, 16, [20, 33, 16, 5], BF16, wide=300)
    _run_and_check(q, cache, table, _int32([20, 33, 16, 5]))
    narrow = table[:, :1].contiguous()
    _run_and_check(q, cache, narrow, _int32([1000, 17, 16, -4]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_pages_not_held(dtype):
    q, cache, table, lengths = _setup(11, 3, 2, 4, 2, 64, 16, [200, 64, 40], dtype)
    table[0, 3:9] = -1
    table[1] = torch.tensor([cache.k.shape[0], -5, 2 ** 31 - 1, -(2 ** 31)] + [-1] * (table.shape[1] - 4), dtype=torch.int32)
    table[2, 2] = -1                                    # the newest tokens' own page
    o, lse = _run_and_check(q, cache, table, lengths)
    assert not bool(o[1].any()) and bool((lse[1] == -math.inf).all())
    _run_and_check(q, cache, table, lengths, window=60, sinks=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_unseen_nan_does_not_reach_a_row(dtype):
    """NaN keys and values in tokens that some rows see and others do not: drafts' futures, window edges."""
    q, cache, table, lengths = _setup(12, 1, 6, 4, 2, 64, 16, [100], dtype)
    nan = torch.full((1, 1, 2, 64), math.nan, device="cuda")
    one = torch.randn(1, 1, 2, 64, generator=_gen(1)).cuda()
    value_nan = one.clone()
    value_nan[..., 5] = math.nan
    kda.cache_write(cache, one, value_nan, table, _int32([97]))          # seen from row 3 on: channel 5
    kda.cache_write(cache, nan, one, table, _int32([98]))                # seen from row 4 on: the whole row
    o, lse = _run_and_check(q, cache, table, lengths)
    assert not bool(torch.isnan(o[:, :3]).any())
    assert bool(torch.isnan(o[:, 3, :, 5]).all()) and not bool(torch.isnan(o[:, 3, :, 6:]).any())
    assert bool(torch.isnan(o[:, 4:]).all()) and bool(torch.isnan(lse[:, 4:]).all())
    kda.cache_write(cache, one, value_nan, table, _int32([88]))          # leaves the window from row 4 on
    q, cache, table, lengths = _setup(13, 1, 6, 4, 2, 64, 16, [100], dtype)
    kda.cache_write(cache, one, value_nan, table, _int32([88]))
    o, _ = _run_and_check(q, cache, table, lengths, window=10, sinks=2)
    assert bool(torch.isnan(o[:, :4, :, 5]).all()) and not bool(torch.isnan(o[:, 4:]).any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("factor", [1.0, 40.0, 1e-3])
def test_attention_uneven_scales(dtype, factor):
    """Pages whose values differ by 2^60 in size, large scores, tiny queries."""
    g = _gen(14)
    heads, d, page, T = 2, 64, 16, 160
    cache, table = kda.cache_new(10, heads, page, d), _table(g, 1, 10, 10).cuda()
    size = torch.exp2(6.0 * torch.randperm(10, generator=g) - 30.0).repeat_interleave(page)[None, :, None, None]
    k, v = (torch.randn(1, T, heads, d, generator=g) for _ in range(2))
    kda.cache_write(cache, k.cuda(), (v * size).cuda(), table, _int32([0]))
    q = (torch.randn(1, 2, 4, d, generator=g) * factor).to(dtype).cuda()
    _run_and_check(q, cache, table, _int32([T]))
    kda.cache_write(cache, (k * size.sqrt()).cuda(), v.cuda(), table, _int32([0]))
    _run_and_check(q, cache, table, _int32([T]), scale=1e-4)


def test_attention_extreme_queries():
    """bf16 queries far outside fp16's range, whole rows of zeros, infinities."""
    q, cache, table, lengths = _setup(15, 1, 4, 2, 1, 64, 16, [50], BF16, spread=0)
    q[0, 0] *= 2.0 ** 100
    q[0, 1] *= 2.0 ** -100
    q[0, 2] = 0
    _run_and_check(q[:, :3].contiguous(), cache, table, lengths, scale=2.0 ** -100)
    # (row 0 left out: its scores would pass 2^190, and scores are 32-bit numbers)
    _run_and_check(q[:, 1:3].contiguous(), cache, table, lengths, scale=2.0 ** 90)
    q[0, 3, 0, 3] = math.inf
    o = kda.cache_attention(q, cache, table, lengths)
    assert bool(torch.isnan(o[0, 3, 0]).all()) and bool(torch.isfinite(o[0, 3, 1]).all())


@pytest.mark.parametrize("B, T_q, hq, hk, d, page, lengths", [
    (1, 8, 4, 1, 128, 64, [100]), (1, 17, 1, 1, 128, 16, [17]), (2, 5, 8, 2, 80, 32, [128, 129]),
    (3, 9, 6, 2, 96, 16, [0, 3, 300]), (1, 16, 8, 2, 112, 128, [1000]), (2, 33, 2, 1, 128, 64, [33, 500]),
    (1, 3, 130, 1, 128, 256, [257]), (1, 70, 3, 1, 128, 16, [70]), (2, 20, 4, 4, 128, 32, [127, 641]),
])
def test_attention_many_rows(B, T_q, hq, hk, d, page, lengths):
    """More than 16 rows a head, bf16, wide heads: the kernel whose codes are operands as they lie."""
    _run_and_check(*_setup(sum(lengths) + d + hq, B, T_q, hq, hk, d, page, lengths, BF16))


@pytest.mark.parametrize("window, sinks", [(1, 1), (16, 4), (100, 17), (129, 0), (64, 300), (1000, 3)])
def test_attention_many_rows_window(window, sinks):
    _run_and_check(*_setup(window + sinks, 2, 12, 4, 2, 128, 16, [12, 777], BF16), window=window, sinks=sinks)


def test_attention_many_rows_long():
    q, cache, table, lengths = _setup(31, 2, 8, 4, 1, 128, 64, [9001, 4096], BF16)
    _run_and_check(q, cache, table, lengths)
    _run_and_check(q, cache, table, lengths, window=5000, sinks=5)


def test_attention_many_rows_many_sequences():
    lengths = [(i * 37) % 300 for i in range(50)]
    q, cache, table, _ = _setup(32, 50, 6, 6, 2, 128, 16, lengths, BF16, wide=60)
    _run_and_check(q, cache, table, _int32(lengths))


def test_attention_many_rows_pages_not_held():
    q, cache, table, lengths = _setup(33, 3, 9, 4, 2, 128, 16, [700, 64, 40], BF16)
    table[0, 3:9] = -1
    table[0, 20:36] = cache.k.shape[0]
    table[1] = -1
    table[2, 2] = -1
    o, lse = _run_and_check(q, cache, table, lengths)
    assert not bool(o[1].any()) and bool((lse[1] == -math.inf).all())
    _run_and_check(q, cache, table, lengths, window=60, sinks=20)


def test_attention_many_rows_unseen_nan():
    q, cache, table, lengths = _setup(34, 1, 12, 4, 2, 128, 16, [300], BF16)
    nan = torch.full((1, 1, 2, 128), math.nan, device="cuda")
    one = torch.randn(1, 1, 2, 128, generator=_gen(1)).cuda()
    value_nan = one.clone()
    value_nan[..., 5] = math.nan
    value_nan[..., 100] = math.nan
    kda.cache_write(cache, one, value_nan, table, _int32([294]))         # seen from row 6 on: two channels
    kda.cache_write(cache, nan, one, table, _int32([297]))               # seen from row 9 on: the whole row
    o, lse = _run_and_check(q, cache, table, lengths)
    assert not bool(torch.isnan(o[:, :6]).any()) and bool(torch.isnan(o[:, 9:]).all())
    assert bool(torch.isnan(o[:, 6:9, :, [5, 100]]).all()) and not bool(torch.isnan(o[:, 6:9, :, 6:100]).any())
    q, cache, table, lengths = _setup(35, 1, 12, 4, 2, 128, 16, [300], BF16)
    kda.cache_write(cache, one, value_nan, table, _int32([275]))         # leaves the window from row 7 on
    o, _ = _run_and_check(q, cache, table, lengths, window=20, sinks=2)
    assert bool(torch.isnan(o[:, :7, :, 5]).all()) and not bool(torch.isnan(o[:, 7:]).any())
    q[0, 3, 1, 7] = math.nan
    o = kda.cache_attention(q, cache, table, lengths)
    assert bool(torch.isnan(o[0, 3, 1]).all()) and not bool(torch.isnan(o[0, :, 0, 6:100]).any())


@pytest.mark.parametrize("factor", [1.0, 40.0, 1e-3])
def test_attention_many_rows_uneven_scales(factor):
    g = _gen(36)
    heads, d, page, T = 2, 128, 16, 320
    cache, table = kda.cache_new(20, heads, page, d), _table(g, 1, 20, 20).cuda()
    size = torch.exp2(3.0 * torch.randperm(20, generator=g) - 30.0).repeat_interleave(page)[None, :, None, None]
    k, v = (torch.randn(1, T, heads, d, generator=g) for _ in range(2))
    kda.cache_write(cache, k.cuda(), (v * size).cuda(), table, _int32([0]))
    q = (torch.randn(1, 10, 4, d, generator=g) * factor).to(BF16).cuda()
    _run_and_check(q, cache, table, _int32([T]))
    kda.cache_write(cache, (k * size.sqrt()).cuda(), v.cuda(), table, _int32([0]))
    _run_and_check(q, cache, table, _int32([T]), scale=1e-4)


def test_attention_many_rows_in_a_row():
    """The same call three times over other work, with strided queries and a workspace of garbage: the same bits."""
    q, cache, table, lengths = _setup(37, 3, 11, 8, 2, 128, 32, [700, 90, 2000], BF16)
    want, want_lse = _run_and_check(q, cache, table, lengths)
    qkv = torch.randn(3, 11, 12 * 128, device="cuda").to(BF16)
    view = qkv[..., : 8 * 128].unflatten(-1, (8, 128))
    view.copy_(q)
    need = kda.cache_attention_workspace_size(3, 11, 8, 2, 128, 32, table.shape[1])
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o, lse = kda.cache_attention(view, cache, table, lengths, workspace=ws, return_lse=True)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_attention_strides_streams_and_buffers():
    q, cache, table, lengths = _setup(16, 2, 3, 8, 2, 64, 32, [700, 90], BF16)
    want, want_lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    qkv = torch.randn(2, 3, 12 * 64, device="cuda").to(BF16)
    view = qkv[..., : 8 * 64].unflatten(-1, (8, 64))
    view.copy_(q)
    out, lse = torch.empty_like(q), torch.empty_like(want_lse)
    need = kda.cache_attention_workspace_size(2, 3, 8, 2, 64, 32, table.shape[1])
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            kda.cache_attention(view, cache, table, lengths, out=out, lse=lse, workspace=ws[:max(need, 1)])
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_step_in_a_graph():
    """Rotary, write and attention captured once and replayed over a growing sequence."""
    g = _gen(17)
    B, hq, hk, d, page, T = 2, 8, 2, 64, 16, 40
    table = _table(g, B, 3, 6).cuda()
    freq = kda.rotary_frequencies(d)
    x = [torch.randn(T, B, 1, n, d, generator=g).to(BF16).cuda() for n in (hq, hk, hk)]

    def step(cache, q, k, v, at):
        q, k = kda.rotary(q, k, at, freq)
        kda.cache_write(cache, k, v, table, at.view(-1))
        return kda.cache_attention(q, cache, table, at.view(-1) + 1)

    eager, graphed = kda.cache_new(6, hk, page, d), kda.cache_new(6, hk, page, d)
    at = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    held = [t[0].clone() for t in x]
    step(graphed, *held, at)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(graphed, *held, at)
    for t in range(T):
        at.fill_(t)
        for h, source in zip(held, x):
            h.copy_(source[t])
        graph.replay()
        want = step(eager, *(s[t] for s in x), at)
        assert torch.equal(o, want), t


@pytest.mark.parametrize("dtype, T_q, d", [(BF16, 1, 64), (F32, 2, 128), (BF16, 9, 128)])
def test_scales_of_a_caller(dtype, T_q, d):
    """Pools that were filled elsewhere: scales that are no powers of two, read, attended over and appended to."""
    g = _gen(20)
    cache, table = _filled(g, 8, 2, 16, d), _table(g, 1, 7, 8)
    for name in "kv":
        codes = getattr(cache, name).view(torch.uint8)
        codes.masked_fill_((codes & 0x7F) == 0x7F, 0x22)                 # no NaN
        getattr(cache, name + "_scale").mul_(1.0 + torch.rand(8, 2, generator=g).cuda())
    n = 100
    q = torch.randn(1, T_q, 4, d, generator=g).to(dtype).cuda()
    _run_and_check(q, cache, table.cuda(), _int32([n]), scale=1e-3)
    rows = torch.stack([ref.Cache(cache).values("k", table, 0, t) for t in range(n)])
    assert torch.equal(kda.cache_read(cache, table.cuda(), _int32([0]), n, dtype=F32)[0][0].cpu(), rows.float())
    x = torch.randn(1, 3, 2, d, generator=g).to(dtype).cuda() * 2.0 ** -20
    before = ref.Cache(cache)
    kda.cache_write(cache, x, x, table.cuda(), _int32([n]))
    after = ref.Cache(cache)
    for h in range(2):
        p, old = int(table[0, n // 16]), float(before.scale["k"][int(table[0, n // 16]), h])
        new = 2.0 ** math.ceil(math.log2(old))
        assert float(after.scale["k"][p, h]) == new
        moved = ref.to_e4m3((before.codes["k"][p, h, : n % 16].float() * torch.tensor(old / new)).double())
        assert torch.equal(after.codes["k"][p, h, : n % 16], moved)


@pytest.mark.parametrize("T_q, d", [(1, 64), (3, 128), (10, 128)])
def test_split_attention_in_a_graph(T_q, d):
    """Work shared out and joined, captured once, replayed over other lengths."""
    q, cache, table, lengths = _setup(21, 3, T_q, 4, 2, d, 16, [2000, 1500, 700], BF16)
    kda.cache_attention(q, cache, table, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
    for now in ([2000, 1500, 700], [17, 0, 699], [1999, 1, 300]):
        lengths.copy_(_int32(now))
        graph.replay()
        want, want_lse = kda.cache_attention(q, cache, table, lengths, return_lse=True)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 code bytes, its far end in use."""
    heads, page, d = 8, 64, 128
    n_pages = (1 << 32) // (heads * page * d) + 40
    k = torch.empty(n_pages, heads, page, d, dtype=torch.uint8, device="cuda")
    codes = k.view(torch.float8_e4m3fn)                  # keys and values may share a pool in a test
    scale = torch.ones(2, n_pages, heads, device="cuda")
    v = torch.empty_like(k).view(torch.float8_e4m3fn)
    cache = kda.PagedCache(codes, v, scale[0], scale[1])
    g = _gen(18)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 3, n_pages - 2]], dtype=torch.int32)
    x = [torch.randn(1, 200, heads, d, generator=g).cuda() for _ in range(2)]
    kda.cache_write(cache, x[0], x[1], table.cuda(), _int32([0]))
    q = torch.randn(1, 2, 16, d, generator=g).to(BF16).cuda()
    o, lse = kda.cache_attention(q, cache, table.cuda(), _int32([200]), return_lse=True)
    back = kda.cache_read(cache, table.cuda(), _int32([0]), 200, dtype=F32)
    used = table[0].long().cuda()                        # the same tokens in a small pool
    small = kda.PagedCache(*(t.view(torch.uint8)[used].view(torch.float8_e4m3fn) for t in cache[:2]), *(t[used] for t in cache[2:]))
    order = _int32([[0, 1, 2, 3]])
    want, want_lse = kda.cache_attention(q, small, order, _int32([200]), return_lse=True)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    for a, b in zip(back, kda.cache_read(small, order, _int32([0]), 200, dtype=F32)):
        assert torch.equal(a, b)
    _check_attention(q, small, order, _int32([200]), o, lse)


def test_binding_refusals():
    q, cache, table, lengths = _setup(19, 2, 1, 4, 2, 64, 16, [20, 30], BF16)
    k = torch.zeros(2, 1, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        kda.cache_attention(q, cache, table.long(), lengths)
    with pytest.raises(ValueError):
        kda.cache_attention(q, cache, table[:1], lengths)
    with pytest.raises(ValueError):
        kda.cache_attention(q[..., :32], cache, table, lengths)
    with pytest.raises(kda.KDAError):                   # one head beside the cache's two
        kda.cache_attention(q.transpose(1, 2), cache, table, lengths)
    with pytest.raises(TypeError):
        kda.cache_attention(q.half(), cache, table, lengths)
    with pytest.raises(ValueError, match="overlap"):
        kda.cache_attention(q[:1].expand(2, 1, 4, 64), cache, table, lengths)
    with pytest.raises(ValueError, match="overlap"):
        kda.rotary(q[:1].expand(2, 1, 4, 64), None, lengths, kda.rotary_frequencies(64))
    with pytest.raises(ValueError, match="evenly"):
        kda.rotary(torch.zeros(2, 5, 2, 64, device="cuda")[:, :3], None, torch.zeros(6, dtype=torch.int32, device="cuda"),
                   kda.rotary_frequencies(64))
    with pytest.raises(kda.KDAError):
        kda.cache_attention(q, cache, table, lengths, window=-1)
    with pytest.raises(ValueError):
        kda.cache_write(cache, k[:, :, :1], k[:, :, :1], table, lengths)
    with pytest.raises(TypeError):
        kda.cache_write(cache, k, k.float(), table, lengths)
    with pytest.raises(ValueError):
        kda.cache_write(cache, k, k, table, lengths, cu_seqlens=_int32([0, 1, 2]))
    with pytest.raises(ValueError):
        kda.rotary(k, None, lengths[:1], kda.rotary_frequencies(64))
    with pytest.raises(TypeError):
        kda.rotary(k, None, lengths, kda.rotary_frequencies(64).float())
