"""Sequences that are cut inside a page that others hold too, and go on: the others keep their tokens, bit for bit."""
import random

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def counted(refs, table):
    return torch.bincount(table[table >= 0].long(), minlength=refs.numel()).to(torch.int32)


def tokens_of(pool, table, row, n, dtype=torch.float32):
    """Keys and values of a row's first n tokens, as they are read."""
    return [x[0] for x in kda.cache_read(pool, table[row: row + 1], ints([0]), n, dtype=dtype)]


@pytest.mark.parametrize("page, heads, d", [(16, 2, 64), (64, 1, 128)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_rows_part_by_forking_to_rows_that_hold_nothing(page, heads, d, seed):
    """Eight forks of three prompts, some cut back to inside their shared pages: forked once more to spare rows, the page copied, the old
    rows given back, then written to, with values so large that the pages' scales grow."""
    rng = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    rows, spare, wide = 11, 8, 12
    n_pages = 19 * wide
    pool = kda.cache_new(n_pages, heads, page, d)
    refs, table, lengths = ints([0] * n_pages), ints([[-1] * wide] * (rows + spare)), ints([0] * (rows + spare))
    prompts = [rng.randint(3 * page, 8 * page) for _ in range(3)]
    kda.cache_resize(refs, table, ints([0, 1, 2]), ints(prompts), page)
    for r, n in enumerate(prompts):
        kda.cache_write(pool, randn(1, n, heads, d), randn(1, n, heads, d), table[r: r + 1], ints([0]))
    lengths[:3] = ints(prompts)
    a, b, missing = kda.cache_fork(refs, table, lengths, ints([i % 3 for i in range(8)]), ints(list(range(3, 11))), page)
    kda.cache_copy(pool, a, b)
    assert int(missing) == 0
    before = {r: tokens_of(pool, table, r, int(lengths[r])) for r in range(rows)}

    cut = rng.sample(range(rows), 6)
    at = [rng.randint(1, int(lengths[r])) for r in cut]
    at[0] = at[0] // page * page + 1                       # a page's first token
    at[1] = max(1, at[1] // page) * page                   # whole pages: nothing to part from
    at[0] = min(at[0], int(lengths[cut[0]]))
    lengths[cut] = ints(at)
    to = rng.sample(range(rows, rows + spare), 6)
    a, b, missing = kda.cache_fork(refs, table, lengths, ints(cut), ints(to), page)
    kda.cache_copy(pool, a, b)
    kda.cache_resize(refs, table, ints(cut), ints([0] * 6), page)
    assert int(missing) == 0 and lengths[to].tolist() == at
    grown = ints([n + 2 * page + 3 for n in at])
    assert int(kda.cache_resize(refs, table, ints(to), grown, page)) == 0
    assert torch.equal(refs, counted(refs, table))
    for r, n in zip(to, at):                               # nothing that is written to has another holder
        assert bool((refs[table[r, n // page: -(-int(n + 2 * page + 3) // page)].long()] == 1).all())
    new = [1000 * randn(1, 2 * page + 3, heads, d) for _ in range(12)]
    for i, (r, n) in enumerate(zip(to, at)):
        kda.cache_write(pool, new[2 * i], new[2 * i + 1], table[r: r + 1], ints([n]))

    for r in range(rows):
        if r not in cut:
            for got, want in zip(tokens_of(pool, table, r, int(lengths[r])), before[r]):
                assert torch.equal(got, want)
    for i, (r, n) in enumerate(zip(to, at)):
        full = n // page * page
        for x, (got, want) in enumerate(zip(tokens_of(pool, table, r, n + 2 * page + 3), before[cut[i]])):
            assert torch.equal(got[:full], want[:full])
            # in the page that the new tokens share, e4m3 at the scale that they brought, below 2 / 448 of its largest value (read with half a
            # step less): half a step of the value, or of the smallest
            page_max = got[full: full + page].abs().amax((0, 2))[:, None] if n % page else torch.zeros(heads, 1, device=DEV)
            off = (got[full: n] - want[full: n]).abs()
            assert bool((off <= 2.0 ** -4 * want[full: n].abs() + 2.0 ** -10 * page_max * 2.14 / 448).all())
            rest = new[2 * i + x][0]
            of_page = torch.cat([got[:n], rest]).abs()     # (a bound on the page's largest value)
            assert bool(((got[n:] - rest).abs() <= 2.0 ** -4 * rest.abs() + 2.0 ** -10 * of_page.max() * 2 / 448 + 1e-30).all())


def test_a_branch_from_an_earlier_token():
    """What fork takes of a source is what the lengths it is given say: a copy of them takes less than the sequence has."""
    page, n_pages = 16, 40
    pool = kda.cache_new(n_pages, 1, page, 64)
    refs, table = ints([0] * n_pages), ints([[-1] * 8] * 4)
    x = torch.randn(1, 100, 1, 64, device=DEV)
    kda.cache_resize(refs, table, ints([0]), ints([100]), page)
    kda.cache_write(pool, x, x, table[:1], ints([0]))
    lengths = ints([100, 0, 0, 0])
    for row, n in ((1, 70), (2, 48), (3, 3)):
        cut = lengths.clone()
        cut[0] = n
        a, b, missing = kda.cache_fork(refs, table, cut, ints([0]), ints([row]), page)
        kda.cache_copy(pool, a, b)
        lengths[row] = cut[row]
        assert int(missing) == 0 and int(lengths[row]) == n and (int(b) >= 0) == (n % page > 0)
        for got, want in zip(tokens_of(pool, table, row, n), tokens_of(pool, table, 0, n)):
            assert torch.equal(got, want)
    assert lengths.tolist() == [100, 70, 48, 3] and torch.equal(refs, counted(refs, table))
