"""Pages of the cache copied, taken and given back, shared by forks and compacted, against lists of Python."""
import random

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Plain:
    """The definitions, an entry after another."""

    def __init__(self, refs, table, page):
        self.refs, self.table, self.page = list(refs), [list(r) for r in table], page
        self.wide = len(table[0]) if table else 0

    def held(self, e):
        return 0 <= e < len(self.refs)

    def free(self):
        return iter([p for p, n in enumerate(self.refs) if n <= 0])

    def resize(self, rows, tokens):
        seen, todo, missing = set(), [], 0
        for r, t in zip(rows, tokens):
            if not 0 <= r < len(self.table) or r in seen:
                continue
            seen.add(r)
            need = min(self.wide, max(0, -(-t // self.page)))
            for j in range(need, self.wide):
                if self.held(self.table[r][j]):
                    self.refs[self.table[r][j]] = max(0, self.refs[self.table[r][j]] - 1)
                self.table[r][j] = -1
            todo += [(r, j) for j in range(need) if not self.held(self.table[r][j])]
        free = self.free()
        for r, j in todo:
            self.table[r][j] = next(free, -1)
            if self.table[r][j] >= 0:
                self.refs[self.table[r][j]] = 1
            else:
                missing += 1
        return missing

    def fork(self, lengths, src, dst):
        copies, ask, missing = [(-1, -1)] * len(src), [], 0
        seen, sources = set(), set(src)
        for i, (a, b) in enumerate(zip(src, dst)):
            earlier = b in seen
            seen.add(b)
            if not (0 <= a < len(self.table) and 0 <= b < len(self.table)) or earlier or b in sources:
                continue
            n = min(max(lengths[a], 0), self.wide * self.page)
            full = n // self.page
            self.table[b] = [e if j < full and self.held(e) else -1 for j, e in enumerate(self.table[a])]
            for e in self.table[b]:
                if e >= 0:
                    self.refs[e] += 1
            if n % self.page and self.held(self.table[a][full]):
                ask.append((i, a, b, full))
            lengths[b] = n
        free = self.free()
        for i, a, b, full in ask:
            p = next(free, -1)
            if p < 0:
                missing += 1
                continue
            self.table[b][full], self.refs[p], copies[i] = p, 1, (self.table[a][full], p)
        return [c[0] for c in copies], [c[1] for c in copies], missing

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        moves = list(zip([p for p in range(n, len(self.refs)) if self.refs[p] > 0], [p for p in range(n) if self.refs[p] <= 0]))
        where = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        refs = [max(r, 0) for r in self.refs]
        for a, b in moves:
            where[a], refs[b], refs[a] = b, refs[a], 0
        self.table = [[where[e] if self.held(e) else -1 for e in row] for row in self.table]
        self.refs = refs
        return where, moves, n


def scattered(rng, n_pages, n_rows, wide, fill, share=0.3):
    """A table whose rows hold about `fill` of their entries, some of them the same pages, and the counts that match it."""
    table = [[-1] * wide for _ in range(n_rows)]
    free = list(range(n_pages))
    rng.shuffle(free)
    refs = [0] * n_pages
    for r in range(n_rows):
        for j in range(rng.randint(0, int(wide * fill))):
            if r and rng.random() < share and table[r - 1][j] >= 0:
                p = table[r - 1][j]
            elif free:
                p = free.pop()
            else:
                continue
            table[r][j] = p
            refs[p] += 1
    return refs, table


# (lists of more than 1,024 rows go another way, and so do warps with more than 1,024 pages)
SIZES = [(400_000, 6, 40), (1, 1, 1), (7, 3, 5), (40, 9, 31), (100, 33, 32), (1000, 20, 257), (5000, 70, 300), (40001, 130, 300), (9000, 1, 9000), (300, 9001, 1),
         (30000, 300, 400), (20000, 1500, 90),           # (calls of more than 65,536 entries)
         (200, 16000, 1), (3000, 8193, 2)]               # (more rows than one CTA counts, little else to look through)


@pytest.mark.parametrize("n_pages, n_rows, wide", SIZES)
@pytest.mark.parametrize("page", [16, 256])
def test_resize(n_pages, n_rows, wide, page):
    rng = random.Random(n_pages + page)
    refs, table = scattered(rng, n_pages, n_rows, wide, 0.8)
    table[0][0] = n_pages                                  # an entry that holds nothing, as -1 does
    plain = Plain(refs, table, page)
    t_refs, t_table = ints(refs), ints(table)
    for step in range(3):
        n = rng.randint(1, n_rows + 2) if n_rows > 1024 else min(rng.randint(1, n_rows + 2), 300)
        rows = [rng.randint(-1, n_rows) for _ in range(n)]  # outside, and some of them twice
        tokens = [rng.choice([0, -5, 1, page, page + 1, rng.randint(0, wide * page + 40), 2 ** 31 - 1]) for _ in range(n)]
        missing = kda.cache_resize(t_refs, t_table, ints(rows), ints(tokens), page)
        assert int(missing) == plain.resize(rows, tokens)
        assert t_table.tolist() == plain.table
        assert t_refs.tolist() == plain.refs
    everything = list(range(n_rows))
    for first in range(0, n_rows, 65536):
        kda.cache_resize(t_refs, t_table, ints(everything), ints([0] * n_rows), page)
    assert int((t_table != -1).sum()) == 0
    plain.resize(everything, [0] * n_rows)
    assert t_refs.tolist() == plain.refs


def test_resize_of_counts_that_do_not_match():
    """A page that the table holds more often than its count says: the count stops at 0."""
    refs, table = ints([1, 0, 2]), ints([[0, 0, 1], [2, -1, -1]])
    kda.cache_resize(refs, table, ints([0]), ints([0]), 16)
    assert refs.tolist() == [0, 0, 2] and table.tolist() == [[-1, -1, -1], [2, -1, -1]]


@pytest.mark.parametrize("n_pages, n_rows, wide", [(12, 6, 3), (100, 33, 32), (3000, 70, 300), (300, 600, 2), (50, 8, 1), (4000, 5000, 3), (9000, 3000, 17),
                                                   (30000, 700, 300), (60000, 3000, 60), (100, 19000, 1), (100, 16500, 0)])
def test_fork(n_pages, n_rows, wide):
    page = 32
    rng = random.Random(n_pages)
    for step in range(4):
        refs, table = scattered(rng, n_pages, n_rows, wide, 1.0)
        half = max(1, n_rows // 2)
        lengths = [rng.choice([0, page, rng.randint(0, wide * page), wide * page + 7, -3]) for _ in range(n_rows)]
        for r in range(half, n_rows):                      # rows that hold nothing
            for j in range(wide):
                if table[r][j] >= 0:
                    refs[table[r][j]] -= 1
                table[r][j] = -1
        n = rng.randint(1, n_rows)
        src = [rng.randint(-1, half - 1) for _ in range(n)]
        dst = [rng.randint(half, n_rows) for _ in range(n)]  # some of them twice, some outside
        if step == 3 and n > 1:
            dst[0] = src[-1]                               # a source
        plain, t_refs, t_table, t_lengths = Plain(refs, table, page), ints(refs), ints(table), ints(lengths)
        got = kda.cache_fork(t_refs, t_table, t_lengths, ints(src), ints(dst), page)
        want = plain.fork(lengths, src, dst)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and int(got[2]) == want[2]
        assert t_table.tolist() == plain.table and t_refs.tolist() == plain.refs and t_lengths.tolist() == lengths


@pytest.mark.parametrize("n_pages, n_rows, wide", SIZES)
def test_compact(n_pages, n_rows, wide):
    rng = random.Random(n_pages)
    for fill in (0.0, 0.2, 1.0):
        refs, table = scattered(rng, n_pages, n_rows, wide, fill)
        table[0][0] = -7 if table[0][0] < 0 else table[0][0]
        if n_pages > 3:
            refs[n_pages - 2] += 1                         # held by something else than the table
            refs[1] -= 2 if refs[1] == 0 else 0            # a count below 0 is none
        plain, t_refs, t_table = Plain(refs, table, 16), ints(refs), ints(table)
        where, moves, held = plain.compact()
        out_refs, out_table = torch.full_like(t_refs, 99), torch.full_like(t_table, 99)
        kda.cache_compact(t_refs, t_table, refs_out=out_refs, table_out=out_table)
        assert t_refs.tolist() == refs and t_table.tolist() == table
        got = kda.cache_compact(t_refs, t_table)
        assert got[0].tolist() == where and int(got[3]) == held
        rest = [-1] * (n_pages // 2 - len(moves))
        assert got[1].tolist() == [a for a, _ in moves] + rest and got[2].tolist() == [b for _, b in moves] + rest
        for r, t in ((t_refs, t_table), (out_refs, out_table)):
            assert r.tolist() == plain.refs and t.tolist() == plain.table


def random_pool(n_pages, heads, page, d, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pool = kda.cache_new(n_pages, heads, page, d)
    for name in "kv":
        getattr(pool, name).view(torch.uint8).copy_(torch.randint(0, 256, (n_pages, heads, page, d), generator=g, device=DEV, dtype=torch.uint8))
        getattr(pool, name + "_scale").copy_(torch.rand(n_pages, heads, generator=g, device=DEV))
    return pool


def bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


@pytest.mark.parametrize("heads, page, d", [(1, 16, 16), (2, 16, 64), (3, 64, 48), (8, 64, 128), (1, 256, 128), (5, 128, 80)])
@pytest.mark.parametrize("n", [1, 6, 33])
def test_copy(heads, page, d, n):
    n_pages = 80
    pool = random_pool(n_pages, heads, page, d)
    rng = random.Random(n)
    ids = rng.sample(range(n_pages), 2 * n)
    src, dst = ids[:n], ids[n:]
    if n > 2:
        src[1], dst[2] = -1, n_pages                       # pairs that are skipped
        src[3] = src[4] = src[0]                           # one page to several
        dst[5] = src[5]                                    # onto itself
    want = [bits(x).clone() for x in pool]
    for a, b in zip(src, dst):
        if 0 <= a < n_pages and 0 <= b < n_pages:
            for w in want:
                w[b] = w[a]
    assert kda.cache_copy(pool, ints(src), ints(dst)) is pool
    for w, x in zip(want, pool):
        assert torch.equal(w, bits(x))


def test_copy_beyond_32_bits():
    """Pages whose bytes begin past 2^32 (a pool of 5.4 GB for keys and as much for values)."""
    n_pages = 41000
    pool = kda.cache_new(n_pages, 8, 128, 128)
    last = n_pages - 1
    bits(pool.k)[last].fill_(7)
    bits(pool.v)[5].fill_(9)
    pool.k_scale[last].fill_(0.25)
    kda.cache_copy(pool, ints([last, 5]), ints([2, last - 1]))
    assert int((bits(pool.k)[2] != 7).sum()) == 0 and int((bits(pool.v)[last - 1] != 9).sum()) == 0
    assert pool.k_scale[2].tolist() == [0.25] * 8


def test_calls_in_a_graph_and_on_another_stream():
    page, n_pages, rows, wide = 16, 500, 12, 20
    refs, table, lengths = ints([0] * n_pages), ints([[-1] * wide] * rows), ints([0] * rows)
    pool = random_pool(n_pages, 2, page, 32)
    all_rows, tokens, src, dst = ints(list(range(rows))), ints([0] * rows), ints([0] * 4), ints([5, 6, 7, 8])

    def step():
        kda.cache_resize(refs, table, all_rows, tokens, page)
        lengths.copy_(tokens)
        a, b, _ = kda.cache_fork(refs, table, lengths, src, dst, page)
        kda.cache_copy(pool, a, b)
        page_map, c, d, held = kda.cache_compact(refs, table)
        kda.cache_copy(pool, c, d)
        return held

    def expected(token_list, plain, codes):
        plain.resize(list(range(rows)), token_list)
        n = list(token_list)
        for a, b in zip(*plain.fork(n, [0] * 4, [5, 6, 7, 8])[:2]):
            if a >= 0:
                codes[b] = codes[a]
        for a, b in plain.compact()[1]:
            codes[b] = codes[a]

    plain, codes = Plain(refs.tolist(), table.tolist(), page), bits(pool.k).cpu().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    expected([0] * rows, plain, codes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = random.Random(3)
    for _ in range(4):
        now = [rng.randint(0, wide * page) for _ in range(5)] + [0] * 7
        now[0] = rng.randint(20, wide * page)
        tokens.copy_(ints(now))
        graph.replay()
        expected(now, plain, codes)
        assert table.tolist() == plain.table and refs.tolist() == plain.refs
        assert torch.equal(bits(pool.k).cpu(), codes)


def test_refusals():
    refs, table, one = ints([0] * 8), ints([[-1] * 4] * 2), ints([0])
    pool = kda.cache_new(8, 2, 16, 32)
    with pytest.raises(ValueError, match="shape"):
        kda.cache_resize(refs, table, one, ints([1, 2]), 16)
    with pytest.raises(TypeError, match="int32"):
        kda.cache_resize(refs.long(), table, one, one, 16)
    with pytest.raises(kda.KDAError, match="a page is"):
        kda.cache_resize(refs, table, one, one, 20)
    with pytest.raises(kda.KDAError, match="workspace"):
        kda.cache_resize(refs, table, one, one, 16, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        kda.cache_fork(refs, ints([[-1] * 4] * 4).T, ints([0] * 4), one, one, 16)
    with pytest.raises(ValueError, match="lengths"):
        kda.cache_fork(refs, table, ints([0] * 3), one, one, 16)
    with pytest.raises(ValueError, match="page_map"):
        kda.cache_compact(refs, table, page_map=ints([0] * 7))
    with pytest.raises(ValueError, match="dst"):
        kda.cache_copy(pool, one, ints([1, 2]))
    # nothing to do
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    kda.cache_copy(pool, none, none)
    assert int(kda.cache_resize(refs, table, none, none, 16)) == 0
    assert int(kda.cache_fork(refs, table, ints([0, 0]), none, none, 16)[2]) == 0
    assert int(kda.cache_compact(none, torch.empty(0, 4, dtype=torch.int32, device=DEV))[3]) == 0
    assert int(kda.cache_resize(none, table, one, ints([40]), 16)) == 3
