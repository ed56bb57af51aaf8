"""Attention of groups of sequences over a prefix that they share, against each sequence's attention over its own row in 64 bits."""
import math
import random
import time

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
# Whether prefixes are taken by themselves follows from the sizes, the prefix table's width among them: "wide" fills that up with
# entries that hold nothing, until they are.
WIDE, WIDE32 = "wide", "wide fp32"
KINDS = [BF16, F32, WIDE, WIDE32]


def room(dtype, sequences, groups, rows, hk, d):
    """Tokens of prefix tables that are enough (fp32 rows that fill their tiles by themselves: none are)."""
    d = 64 if d <= 64 else 128
    tile = 10 if rows <= 8 else 16 if rows <= 16 else 32 if rows <= 32 else -(-rows // 64) * 64
    reads = -(-rows // 32) if dtype == BF16 else (tile - rows) / 8
    saved = reads * (sequences - groups) * hk * 2 * d
    return int(((96 << 20) + (1 if dtype == BF16 else 6) * sequences * rows * hk * 8 * d) / saved) + 1 if saved > 0 else 0


HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """groups: (shared tokens, [tokens of each sequence beyond them]); negative: that many tokens short of the prefix;
    None: a place not in use."""

    def __init__(self, seed, T_q, hq, hk, d, page, dtype, groups, before=(), after=(), spread=3, extra_pages=0, more=0):
        g = torch.Generator().manual_seed(seed)
        shared = [s for s, _ in groups]
        rows = sum(len(own) for _, own in groups) + len(before) + len(after)
        wide, dtype = dtype in (WIDE, WIDE32), {WIDE: BF16, WIDE32: F32}.get(dtype, dtype)
        wide_extra = room(dtype, rows, len(groups), T_q * hq // hk, hk, d) // page + 1 if wide else 0
        lengths, cu, of = list(before), [len(before)], [None] * len(before)
        for i, (s, own) in enumerate(groups):
            lengths += [0 if n is None else max(0, s + n) for n in own]
            of += [i] * len(own)
            cu.append(len(lengths))
        lengths += list(after)
        of += [None] * len(after)
        pages = lambda n: -(-n // page)  # noqa: E731
        n_pages = sum(pages(s) for s in shared) + sum(pages(n) for n in lengths) + 2
        ids = iter(torch.randperm(n_pages, generator=g).tolist())
        wide_prefix = max([pages(s) for s in shared] + [0]) + extra_pages + wide_extra
        wide = max([pages(n) for n in lengths] + [1]) + extra_pages + pages(more)
        prefix = [[next(ids) for _ in range(pages(s))] for s in shared]
        rows = []
        for n, o in zip(lengths, of):
            common = prefix[o][: min(shared[o] // page, pages(n))] if o is not None else []
            rows.append(common + [next(ids) for _ in range(pages(n) - len(common))])
        self.prefix_table = ints([p + [-1] * (wide_prefix - len(p)) for p in prefix]).view(len(groups), wide_prefix)
        self.table = ints([r + [-1] * (wide - len(r)) for r in rows])
        self.lengths, self.shared, self.cu, self.d, self.page = ints(lengths), ints(shared), ints(cu), d, page
        codes, scales = [], []
        for _ in range(2):
            c = torch.randint(0, 0x7F, (n_pages, hk, page, d), generator=g, dtype=torch.uint8)
            c |= torch.randint(0, 2, c.shape, generator=g, dtype=torch.uint8) << 7
            c = torch.where((c & 0x7F) > 0x58, c - 0x20, c)   # few of the very large
            codes.append(c)
            scales.append(torch.exp2(torch.randint(-spread, spread + 1, (n_pages, hk), generator=g).float() - 4))
        last = {}
        for r, n in zip(rows, lengths):                    # what no token was written to is not a number
            if n % page and not any(r[-1] in p for p in prefix):
                last[r[-1]] = n % page
        for p, n in last.items():
            for c in codes:
                c[p, :, n:] = 0x7F
        self.pool = kda.PagedCache(*(c.to(DEV).view(torch.float8_e4m3fn) for c in codes), *(s.to(DEV) for s in scales))
        self.q = (torch.randn(len(lengths), T_q, hq, d, generator=g) * 0.5).to(dtype).to(DEV)

    def run(self, **kw):
        return kda.cache_attention_shared(self.q, self.pool, self.table, self.lengths, self.prefix_table, self.shared, self.cu,
                                          return_lse=True, **kw)

    def check(self, o, lse, scale=None):
        """The bound, as in the tests of cache_attention: scores 2^-24 (2 d + 8) of the sum of |q k|, and what three pieces of fp8
        or less lose of a query: half of 2^-21 of its row's largest value a channel; weights half a step 2^-11 (fp32: two fp16
        numbers, 2^-21), below fp16's normal range 2^-31 of the row's reference a token; exponentials 2^-21, again 2^-20 for the joining's
        factors; sums 2^-24 (n / 16 + 64); products of 64 tiles cut off by at most 512 steps 2^-23 of the sum, 2^-14.  All of
        that twice, for the division; half a step of the output's type."""
        q, d = self.q.double(), self.d
        scale = 1 / math.sqrt(d) if scale is None else scale
        B, t_q, hq, _ = q.shape
        hk = self.pool.k.shape[1]
        values = {n: getattr(self.pool, n).float().double() * getattr(self.pool, n + "_scale").double()[:, :, None, None] for n in "kv"}
        worst = 0.0
        for b in range(B):
            length = min(int(self.lengths[b]), self.table.shape[1] * self.page)
            at = torch.arange(max(length, 0), device=DEV)
            ids = self.table[b].long()[at // self.page] if length > 0 else at
            held = (ids >= 0) & (ids < values["k"].shape[0])
            at, ids = at[held], ids[held]
            for h in range(hk):
                rows = slice(h * hq // hk, (h + 1) * hq // hk)
                qq = q[b, :, rows]                         # [t_q, group, d]
                k, v = (values[n][ids, h, at % self.page] for n in "kv")
                unseen = at > (length - t_q + torch.arange(t_q, device=DEV))[:, None]
                k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
                s = scale * torch.einsum("igd,td->igt", qq, k)
                s = s.masked_fill(unseen[:, None], -math.inf)
                want_lse = torch.logsumexp(s, -1)
                w = torch.exp(s - want_lse[..., None]).nan_to_num(0.0)
                want = w @ v
                weight = w @ v.abs()
                size = (abs(scale) * torch.einsum("igd,td->igt", qq.abs(), k.abs())).amax(-1) if len(at) else torch.zeros(t_q, qq.shape[1], dtype=F64, device=DEV)
                lost = abs(scale) * 2.0 ** -22 * qq.abs().amax(-1) * (k.abs().sum(-1).max() if len(at) else 0.0)
                vs = self.pool.v_scale.double()[ids, h] if len(at) else torch.zeros(0, dtype=F64, device=DEV)
                floor = ((w * vs).amax(-1) if len(at) else torch.zeros_like(size))[..., None] * ((v.abs() / vs[:, None]).sum(0) if len(at) else torch.zeros(d, dtype=F64, device=DEV))
                score = 2.0 ** -24 * (2 * d + 8) * size + lost
                n = max(length, 1)
                step = (2.0 ** -11 if self.q.dtype == BF16 else 2.0 ** -21) + 2.0 ** -20 + 2.0 ** -24 * (n / 16 + 64) + \
                    (2.0 ** -14 if self.q.dtype == BF16 else 0.0)
                tol = HALF_STEP[self.q.dtype] * want.abs() + 2 * (score + step)[..., None] * weight + 2.0 ** -31 * floor + 1e-30
                got, got_lse = o[b, :, rows].double(), lse[b, :, rows].double()
                empty = want_lse == -math.inf
                assert not bool(got[empty].any()) and bool((got_lse[empty] == -math.inf).all())
                err = ((got - want).abs() / tol)[~empty]
                assert bool((err <= 1).all()), (b, h, float(err.max()), int(err.isnan().sum()))
                lse_tol = score + 2.0 ** -20 + 2.0 ** -22 * want_lse.abs() + 2.0 ** -24 * (n / 16 + 64)
                assert bool(((got_lse - want_lse).abs() <= lse_tol)[~empty].all()), float(((got_lse - want_lse).abs() / lse_tol)[~empty].max())
                worst = max(worst, float(err.max()) if err.numel() else 0.0)
        return worst


def both(case, **kw):
    o, lse = case.run(**kw)
    case.check(o, lse, **kw)
    return o, lse


SIZES = [  # T_q, hq, hk, d, page, groups
    (1, 1, 1, 16, 16, [(16, [1, 1])]),
    (1, 8, 2, 64, 16, [(77, [1, 5, 40])]),
    (1, 4, 4, 128, 64, [(64, [0, 1, 2]), (200, [3, 70])]),
    (2, 6, 2, 80, 32, [(100, [2, 3, 40, 31])]),
    (3, 14, 2, 112, 16, [(130, [3, 90]), (16, [4] * 9), (47, [3, 5])]),
    (1, 8, 1, 128, 256, [(513, [1] * 20)]),
    (1, 16, 1, 48, 128, [(300, [7] * 17)]),
    (7, 20, 4, 128, 32, [(500, [7, 9, 200])]),
    (40, 4, 2, 64, 16, [(33, [40, 75, 41])]),
    (33, 8, 2, 128, 64, [(140, [33, 34, 100])]),
    (1, 32, 4, 96, 16, [(129, list(range(1, 40)))]),
    (1, 6, 3, 32, 16, [(40, [(i * 37) % 90 for i in range(30)]), (90, [1, 2]), (15, [1, 2, 3])]),
    (5, 40, 1, 128, 64, [(70, [5, 6, 7])]),
]


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("T_q, hq, hk, d, page, groups", SIZES)
def test_sizes(dtype, T_q, hq, hk, d, page, groups):
    both(Case(d + hq, T_q, hq, hk, d, page, dtype, groups))


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("T_q, group, d", [(1, 2, 64), (1, 8, 128), (3, 4, 128), (12, 3, 80)])
def test_places_not_in_use_and_sequences_that_do_not_see_all(dtype, T_q, group, d):
    """Lengths of 0 (their rows of the table hold nothing), shorter than the prefix, the newest query's token the prefix's last."""
    groups = [(96, [T_q, None, -40, 0, -1, 30, T_q - 1]), (64, [None, None]), (32, [9 + T_q]), (0, [3, 4]), (80, [-79, -80, T_q])]
    both(Case(1, T_q, 2 * group, 2, d, 32, dtype, groups, before=[5, 0, 100], after=[0, 33]))


@pytest.mark.parametrize("dtype", KINDS)
def test_groups_of_all_sizes(dtype):
    groups = [(32 * (1 + i % 3), [1 + (i * j) % 40 for j in range(i)]) for i in (0, 1, 2, 3, 5, 8, 13, 21)]
    both(Case(2, 1, 12, 2, 64, 32, dtype, groups, before=[40], extra_pages=3))


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("d, hq, B", [(128, 8, 3), (64, 4, 40), (128, 32, 20), (96, 4, 130)])
def test_long(dtype, d, hq, B):
    """Long enough to be cut many times over."""
    both(Case(3, 1, hq, 1, d, 64, dtype, [(9001, [1 + 13 * i for i in range(B)])]))


@pytest.mark.parametrize("hk, group, T_q, d, page, n", [(16, 16, 16, 64, 32, 30000), (19, 8, 32, 128, 128, 26001)])
def test_long_for_every_processor(hk, group, T_q, d, page, n):
    """Many rows of many heads: each processor walks more tiles of one prefix than it adds up in one place."""
    both(Case(14, T_q, hk * group, hk, d, page, BF16, [(n, [T_q, T_q + 3, T_q + 90])], spread=1))


@pytest.mark.parametrize("slow", [slice(0, 8), slice(8, 16)])
def test_halves_of_different_speeds(slow):
    """Scores beyond 2^22 take a longer way: 128 of 256 rows that are worked on side by side have them, for many tiles."""
    case = Case(18, 1, 256, 16, 64, 64, BF16, [(20000, [1 + i for i in range(16)])], spread=0)
    case.q[slow] *= 2.0 ** 24
    want = both(case)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(case.run(), want))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T_q, hq, hk, d, n, tokens", [(1, 32, 8, 128, 120, 900), (3, 16, 16, 80, 60, 600), (1, 16, 16, 48, 90, 1000), (38, 16, 4, 128, 30, 1900),
                                                       (2, 32, 32, 64, 40, 1111)])
def test_many_sequences_behind_a_short_prefix(dtype, T_q, hq, hk, d, n, tokens):
    """Sharing pays, and no item is cut."""
    assert 0 < room(dtype, n, 1, T_q * hq // hk, hk, d) <= tokens // 32 * 32
    both(Case(22, T_q, hq, hk, d, 32, dtype, [(tokens, [T_q + i % 37 for i in range(n)])]))


@pytest.mark.parametrize("T_q, hq, hk, d", [(1, 4, 2, 128), (2, 16, 2, 64), (1, 8, 1, 96), (1, 2, 2, 16)])
def test_groups_of_few_rows(T_q, hq, hk, d):
    """bf16 prefixes on the kernels for few rows: up to 16 rows a group, or 32 of 64 channels."""
    both(Case(23, T_q, hq, hk, d, 32, WIDE, [(700 + 90 * i, [T_q + 7 * i, T_q + 50]) for i in range(5)], after=[0, 20]))


@pytest.mark.parametrize("dtype", [WIDE, WIDE32])
def test_prefixes_of_every_length_around_a_tile(dtype):
    """Ends inside, at and behind a tile of 128 tokens, and inside a page; the prefix's last page whole or not."""
    groups = [(s, [1 + (s + i) % 7 for i in range(2 + s % 3)]) for s in (1, 31, 32, 127, 128, 129, 159, 160, 161, 255, 256, 257, 288, 300)]
    both(Case(15, 1, 8, 2, 64, 32, dtype, groups))
    both(Case(16, 1, 4, 1, 128, 256, dtype, groups))


@pytest.mark.parametrize("T_q, hq, hk, d, page, groups", [
    (5, 8, 2, 128, 64, [(64, [5, 6, 300]), (200, [5, 70])]), (40, 4, 2, 80, 16, [(33, [40, 75, 41]), (16, [0, None, -3])]),
    (33, 16, 2, 128, 32, [(140, [33, 34, 2600])]), (3, 14, 2, 112, 16, [(130, [3, 90]), (16, [4] * 9), (47, [3, 1500])])])
@pytest.mark.parametrize("more", [0, 2000])
def test_rests_with_room_for_more(T_q, hq, hk, d, page, groups, more):
    """Which kernel takes the rest of more than 16 rows a head follows from the room behind the prefix."""
    both(Case(19, T_q, hq, hk, d, page, WIDE, groups, before=[50], after=[0], more=more))


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("n", [3, 150])
def test_pages_not_held(dtype, n):
    case = Case(4, 2, 4, 2, 64, 16, dtype, [(400, [2 + i % 30 for i in range(n)])])
    for gone in (3, 4, 5, 17):
        case.prefix_table[0, gone] = -1 if gone != 4 else case.pool.k.shape[0]
        case.table[:, gone] = -1
    case.table[1, 25:] = -1
    both(case)
    case.prefix_table[:] = -1
    case.table[:, :25] = -1
    o, lse = both(case)
    assert bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("factor", [1.0, 40.0, 1e-3])
def test_uneven_scales(dtype, n, factor):
    """Pages whose values differ by 2^60 in size, one after another; large scores, tiny queries."""
    case = Case(5, 1, 4, 2, 64, 16, dtype, [(16 * 30, [1 + i % 40 for i in range(n)])])
    order = torch.randperm(30, generator=torch.Generator().manual_seed(1)).float().to(DEV)
    case.pool.v_scale[case.prefix_table[0, :30].long()] = torch.exp2(2 * order - 30)[:, None]
    case.q *= factor
    both(case)
    case.pool.k_scale[case.prefix_table[0, :30].long()] = torch.exp2(order - 15)[:, None]
    both(case, scale=1e-4)
    both(case, scale=-1e-4)
    both(case, scale=0.0)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("n", [2, 70])
def test_extreme_queries(dtype, n):
    """Far outside fp16's range, rows of zeros, rows without a number."""
    case = Case(6, 3, 4, 2, 128, 32, dtype, [(200, [3 + i % 40 for i in range(n)])], spread=0)
    case.q[:, 0] *= 2.0 ** 100
    case.q[:, 1] = 0
    both(case, scale=2.0 ** -104)
    case.q[:, 0] *= 2.0 ** -200
    both(case, scale=2.0 ** 90)
    clean, clean_lse = case.run(scale=2.0 ** 90)
    case.q[1, 2, 3, 7] = math.nan
    o, lse = case.run(scale=2.0 ** 90)
    mine = torch.zeros_like(lse, dtype=torch.bool)
    mine[1, 2, 3] = True
    assert bool(torch.isnan(o[mine]).all()) and bool(torch.isnan(lse[mine]).all())
    # (rows of a warp move their references together: roundings of the others may differ)
    assert bool(((lse - clean_lse).abs() <= 2.0 ** -20 * clean_lse.abs() + 2.0 ** -9)[~mine].all())
    assert bool(((o.float() - clean.float()).abs() <= 2.0 ** -6 * clean.float().abs().max())[~mine].all())


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("n", [2, 70])
def test_infinite_queries(dtype, n):
    """A channel of -inf against keys of one sign makes every score -inf: 0 and -inf.  +inf, or keys of both signs: no number."""
    case = Case(7, 2, 4, 2, 64, 32, dtype, [(160, [2 + i % 40 for i in range(n)])])
    raw = case.pool.k.view(torch.uint8)
    raw.copy_(torch.where((raw & 0x7F) == 0x7F, raw, (raw & 0x3F) | 0x20))   # positive, not 0
    case.q[1, 1, 2, 5] = -math.inf
    case.q[0, 0, 1, 9] = math.inf
    o, lse = case.run()
    assert not bool(o[1, 1, 2].any()) and float(lse[1, 1, 2]) == -math.inf
    assert bool(torch.isnan(o[0, 0, 1]).all()) and math.isnan(float(lse[0, 0, 1]))
    good = torch.ones_like(lse, dtype=torch.bool)
    good[1, 1, 2] = good[0, 0, 1] = False
    assert bool(torch.isfinite(o[good]).all()) and bool(torch.isfinite(lse[good]).all())
    case.q[:] = -math.inf
    o, lse = case.run()
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    raw[case.prefix_table[0, 2].long()] ^= 0x80            # the prefix's third page: the other sign
    o, lse = case.run()
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("n", [2, 70])
def test_nan_in_the_prefix_reaches_its_channel_only(dtype, n):
    case = Case(8, 1, 4, 2, 64, 32, dtype, [(160, [1 + i % 40 for i in range(n)] + [-130])])
    page = int(case.prefix_table[0, 3])
    case.pool.v.view(torch.uint8)[page, 1, 7, 11] = 0xFF
    o, lse = case.run()
    assert bool(torch.isnan(o[:n, 0, 2:, 11]).all()) and bool(torch.isfinite(lse).all())
    o[:n, 0, 2:, 11] = 0
    assert bool(torch.isfinite(o).all())
    case.pool.k.view(torch.uint8)[page, 0, 7, 11] = 0x7F    # a key: whole rows of head 0
    o, lse = case.run()
    assert bool(torch.isnan(o[:n, 0, :2]).all()) and bool(torch.isnan(lse[:n, 0, :2]).all())
    assert bool(torch.isfinite(lse[:n, 0, 2:]).all()) and bool(torch.isfinite(o[n]).all())


@pytest.mark.parametrize("dtype, T_q, d", [(BF16, 1, 64), (BF16, 2, 128), (WIDE32, 1, 128), (BF16, 40, 80), (WIDE, 1, 64), (WIDE, 40, 80), (WIDE32, 5, 64)])
def test_strides_buffers_and_another_stream(dtype, T_q, d):
    case = Case(9, T_q, 6, 2, d, 16, dtype, [(100, [T_q + i for i in range(9)]), (33, [T_q, 50])])
    dtype = case.q.dtype
    o, lse = both(case)
    fused = torch.full((11, T_q, 10 * d), math.nan, dtype=dtype, device=DEV)
    fused[..., : 6 * d] = case.q.flatten(2)
    q, case.q = case.q, fused[..., : 6 * d].unflatten(-1, (6, d))
    again, lse2 = case.run()
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    need = kda.cache_attention_shared_workspace_size(11, T_q, 6, 2, d, 16, case.table.shape[1], case.prefix_table.shape[1], 2)
    guard = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((13, T_q, 6, d), 7.0, dtype=dtype, device=DEV)
    stats = torch.full((13, T_q, 6), 7.0, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        case.run(out=out[1:12], lse=stats[1:12], workspace=guard[256: 256 + need])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out[1:12], o) and torch.equal(stats[1:12], lse)
    assert bool((out[::12] == 7).all()) and bool((stats[::12] == 7).all())
    assert bool((guard[:256] == 0xA5).all()) and bool((guard[256 + need:] == 0xA5).all())


@pytest.mark.parametrize("dtype, T_q, hq, d", [(BF16, 1, 4, 64), (BF16, 6, 16, 128), (WIDE, 1, 4, 64), (WIDE, 1, 16, 128), (WIDE, 6, 16, 128), (F32, 1, 4, 128), (WIDE32, 1, 4, 128), (WIDE32, 8, 16, 64)])
def test_graph_with_lengths_that_change(dtype, T_q, hq, d):
    """One captured graph, replayed as sequences grow, places come and go, groups change; two graphs with one workspace."""
    case = Case(10, T_q, hq, 2, d, 32, dtype, [(300, [T_q + 40] * 12), (64, [T_q + 60, 90])], after=[50])
    need = kda.cache_attention_shared_workspace_size(15, T_q, hq, 2, d, 32, case.table.shape[1], case.prefix_table.shape[1], 2)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    case.run(workspace=ws)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = case.run(workspace=ws)
        graphs.append((graph, got))
    rng = random.Random(1)
    for step in range(3):
        full = case.lengths.tolist()
        case.lengths.copy_(ints([rng.choice([n, n - rng.randint(0, 30), 0 if step else n]) for n in full]))
        case.shared.copy_(ints([rng.choice([300, 200, 0]), rng.choice([64, 33])]))
        for graph, (o, lse) in graphs:
            graph.replay()
        want = case.run()
        for _, (o, lse) in graphs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        case.check(*want)
        case.lengths.copy_(ints(full))


def test_calls_at_once():
    """Two streams' calls, each with its workspace, beside attention over each row alone."""
    cases = [Case(24 + i, T_q, hq, 2, d, 32, WIDE, [(3000 + 500 * i, [T_q + 3 * j for j in range(40)])]) for i, (T_q, hq, d) in enumerate([(1, 16, 128), (9, 8, 80)])]
    want = [both(c) for c in cases]
    alone = kda.cache_attention(cases[1].q, cases[1].pool, cases[1].table, cases[1].lengths)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for stream, case in zip(streams, cases):
            with torch.cuda.stream(stream):
                got.append(case.run())
        with torch.cuda.stream(streams[2]):
            got.append(kda.cache_attention(cases[1].q, cases[1].pool, cases[1].table, cases[1].lengths))
    torch.cuda.synchronize()
    for i in range(0, len(got), 3):
        for (o, lse), (wo, wl) in zip(got[i: i + 2], want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
        assert torch.equal(got[i + 2], alone)


@pytest.mark.parametrize("dtype, d", [(BF16, 128), (WIDE, 128), (WIDE, 64), (WIDE32, 128)])
def test_pages_beyond_four_gigabytes(dtype, d):
    case = Case(20, 1, 8, 4, d, 256, dtype, [(700, [1 + i for i in range(6)]), (300, [4, 9])])
    want = both(case)
    small, n, more = case.pool, case.pool.k.shape[0], (1 << 32) // (4 * 256 * d) + 100
    case.pool = kda.cache_new(more + n, 4, 256, d)
    for a, b in zip(case.pool, small):
        a.view(torch.uint8 if a.element_size() == 1 else F32)[more:].copy_(b.view(torch.uint8 if b.element_size() == 1 else F32))
    for t in (case.table, case.prefix_table):
        t.copy_(torch.where(t >= 0, t + more, t))
    assert all(torch.equal(a, b) for a, b in zip(case.run(), want))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nearly_two_to_the_31_tokens_mostly_not_held(dtype):
    """The tables' largest sizes, some pages here and there: as attention over these alone."""
    g = torch.Generator(device=DEV).manual_seed(21)
    page, wide, n = 256, (1 << 23) - 1, 7
    pool = kda.cache_new(n, 1, page, 64)
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(dtype)  # noqa: E731
    kda.cache_write(pool, randn(1, n * page, 1, 64), randn(1, n * page, 1, 64), torch.arange(n, device=DEV, dtype=torch.int32)[None], ints([0]))
    places = torch.tensor([0, 12345, 4000001, 8388600, wide - 3, wide - 2, wide - 1], device=DEV)
    table = torch.full((2, wide), -1, dtype=torch.int32, device=DEV)
    table[:, places] = torch.arange(n, device=DEV, dtype=torch.int32)
    q = randn(2, 1, 2, 64)
    prefix = table[:1, : wide - 1].contiguous()
    o, lse = kda.cache_attention_shared(q, pool, table, ints([wide * page - 100] * 2), prefix, ints([(wide - 1) * page]), ints([0, 2]), return_lse=True)
    alone, alone_lse = kda.cache_attention(q, pool, torch.arange(n, device=DEV, dtype=torch.int32).repeat(2, 1), ints([n * page - 100] * 2),
                                           return_lse=True)
    assert bool(((lse - alone_lse).abs() <= 2e-5).all())
    assert bool(((o.float() - alone.float()).abs() <= HALF_STEP[dtype] * 2 * alone.float().abs() + 2.0 ** -9 * (1 if dtype == BF16 else 2.0 ** -6)).all())


def test_no_groups_and_nothing_shared():
    """Without groups, or with nothing to share, it is cache_attention, bit for bit."""
    case = Case(11, 2, 4, 2, 64, 16, BF16, [(0, [5, 60]), (15, [7, 8])], after=[40])
    want = kda.cache_attention(case.q, case.pool, case.table, case.lengths, return_lse=True)
    none = case.prefix_table[:0], case.shared[:0], case.cu[:1]
    for prefix, shared, cu in (none, (case.prefix_table, case.shared, case.cu), (case.prefix_table[:, :0].contiguous(), case.shared, case.cu)):
        got = kda.cache_attention_shared(case.q, case.pool, case.table, case.lengths, prefix, shared, cu, return_lse=True)
        assert all(bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-6).all()) for a, b in zip(got, want))
    for a, b in zip(kda.cache_attention_shared(case.q, case.pool, case.table, case.lengths, *none, return_lse=True), want):
        assert torch.equal(a, b)
    empty = kda.cache_new(0, 2, 16, 64)
    o, lse = kda.cache_attention_shared(case.q, empty, case.table, case.lengths, case.prefix_table, case.shared, case.cu, return_lse=True)
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    o = kda.cache_attention_shared(case.q[:0], case.pool, case.table[:0], case.lengths[:0], *none)
    assert o.shape == (0, 2, 4, 64)


@pytest.mark.parametrize("dtype", KINDS)
def test_malformed_groups_stay_in_the_buffers(dtype):
    case = Case(12, 1, 4, 2, 64, 16, dtype, [(64, [5, 60, 7]), (48, [7, 8])])
    for cu in ([0, 5, 0], [-5, 3, 99], [4, 2, 1], [2 ** 31 - 1, -2 ** 31, 5], [0, 0, 0], [5, 5, 5]):
        case.cu.copy_(ints(cu))
        o, lse = case.run()
        torch.cuda.synchronize()
    case.cu.copy_(ints([0, 3, 5]))
    case.shared.copy_(ints([2 ** 31 - 1, -2 ** 31]))
    case.run()
    torch.cuda.synchronize()


@pytest.fixture
def stall():
    yield kda.selftest_attention_stall
    kda.selftest_attention_stall()


@pytest.mark.parametrize("sequences", [40, 20])            # 160 rows a head, and 80: a stream of them, or both take one
@pytest.mark.parametrize("loads, tiles", [(0, 1 << 24), (1, 1 << 24), (1 << 24, 0)])
def test_bounded_waits_run_out(stall, sequences, loads, tiles):
    """Loads that stop, or products that do, with a limit of 3 ms: the call returns without numbers, and the next is right."""
    case = Case(17, 1, 8, 2, 64, 64, WIDE, [(50000, [1 + i for i in range(sequences)])])
    want, want_lse = case.run()
    torch.cuda.synchronize()
    stall(loads, tiles, 3000)
    start = time.perf_counter()
    o, lse = case.run()
    torch.cuda.synchronize()
    assert time.perf_counter() - start < 20
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
    stall()
    o, lse = case.run()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_refusals():
    case = Case(13, 1, 4, 2, 64, 16, WIDE, [(64, [5, 60, 7])])
    a = dict(q=case.q, cache=case.pool, block_table=case.table, lengths=case.lengths, prefix_table=case.prefix_table,
             prefix_lengths=case.shared, cu_groups=case.cu)
    for change, error, match in [
            (dict(prefix_lengths=ints([1, 2])), ValueError, "prefix_lengths"), (dict(cu_groups=ints([0])), ValueError, "cu_groups"),
            (dict(prefix_table=case.prefix_table.long()), TypeError, "prefix_table"), (dict(q=case.q.half()), TypeError, None),
            (dict(lengths=ints([1])), ValueError, "lengths"), (dict(scale=math.inf), kda.KDAError, "finite"),
            (dict(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)), kda.KDAError, "workspace"),
            (dict(prefix_table=ints([[0]] * 4), prefix_lengths=ints([1] * 4), cu_groups=ints([0, 1, 2, 3, 3])), kda.KDAError, "more groups")]:
        with pytest.raises(error, match=match):
            kda.cache_attention_shared(**{**a, **change})


@pytest.mark.parametrize("dtype, heads, kv_heads, d", [(BF16, 8, 2, 128), (F32, 4, 4, 64)])
def test_a_served_run(dtype, heads, kv_heads, d):
    """A prompt written once, forked, each fork going on by itself, some let go, the pool compacted: attention over the shared
    prefix and over each row alone agree all along."""
    page, rows, wide, n_pages = 32, 10, 12, 90
    g = torch.Generator(device=DEV).manual_seed(3)
    pool = kda.cache_new(n_pages, kv_heads, page, d)
    refs, table, lengths = ints([0] * n_pages), ints([[-1] * wide] * rows), ints([0] * rows)
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(dtype)  # noqa: E731
    prompt = 170
    kda.cache_resize(refs, table, ints([4]), ints([prompt]), page)
    kda.cache_write(pool, randn(1, prompt, kv_heads, d), randn(1, prompt, kv_heads, d), table[4:5], ints([0]))
    lengths[4] = prompt
    targets = ints([0, 1, 2, 3, 5, 6, 7, 8, 9])
    a, b, missing = kda.cache_fork(refs, table, lengths, ints([4] * 9), targets, page)
    kda.cache_copy(pool, a, b)
    assert int(missing) == 0 and lengths.tolist() == [prompt] * 10
    held = ints([prompt // page * page])
    for step in range(70):
        new = 1 + 2 * (step % 2)
        if step == 40:                                     # half of the rows go, the rest moves together
            gone = ints([0, 2, 5, 9])
            kda.cache_resize(refs, table, gone, ints([0] * 4), page)
            lengths[gone.long()] = 0
            page_map, a, b, n = kda.cache_compact(refs, table)
            kda.cache_copy(pool, a, b)
            assert int((refs > 0).sum()) == int(n) and bool((refs[: int(n)] > 0).all())
        alive = lengths > 0
        start, lengths = lengths, torch.where(alive, lengths + new, lengths)
        everyone = torch.arange(rows, dtype=torch.int32, device=DEV)
        assert int(kda.cache_resize(refs, table, everyone, lengths, page)) == 0
        kda.cache_write(pool, randn(rows, new, kv_heads, d), randn(rows, new, kv_heads, d), table, start)
        q = randn(rows, new, heads, d)
        prefix = torch.nn.functional.pad(table[4:5, : prompt // page], (0, room(dtype, rows, 1, new * heads // kv_heads, kv_heads, d) // page + 1), value=-1)
        o, lse = kda.cache_attention_shared(q, pool, table, lengths, prefix, held, ints([0, rows]), return_lse=True)
        alone, alone_lse = kda.cache_attention(q, pool, table, lengths, return_lse=True)
        assert bool(((lse - alone_lse).abs()[alive] <= 2e-5).all())
        assert bool(((o.float() - alone.float()).abs() <= HALF_STEP[dtype] * 2 * alone.float().abs() + 2.0 ** -9 * (1 if dtype == BF16 else 2.0 ** -6)).all())
        assert not bool(o[~alive].any())
    kda.cache_resize(refs, table, everyone, torch.zeros_like(everyone), page)
    assert not bool(refs.any()) and bool((table == -1).all())
