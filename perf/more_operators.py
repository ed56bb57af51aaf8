"""Cases for measuring what a server does with sequences that share pages of the paged cache.

Five operators, in plain torch (``own`` false) or through this package (``own`` true):

  copy     whole pages of the pool copied to other pages
  resize   rows of the block table brought to the pages that their tokens need: pages taken where the pool
           is free, given back where no row of the table holds them any more
  fork     rows that start as another row's sequence: its full pages shared, its last, partly filled one copied
  compact  all held pages brought to the front of the pool, and the block table with them
  attend   attention for sequences in groups that share a long prefix, which is computed once for each group

A case is a dict of plain values; every random number comes from the seed.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # A handful of pages of a narrow layer, as when a few sequences are about to write to pages they share.
        dict(name="copy few", op="copy", n=3, pool=64, kv_heads=2, d=64, page=16),
        # The pages of a whole batch moved to other places, two gigabytes of them read and written.
        dict(name="copy many", op="copy", n=8192, pool=20000, kv_heads=8, d=128, page=64),
        # Draft tokens of a small batch: the few pages for them taken, and given back when they are rejected.
        dict(name="resize step", op="resize", rows=9, listed=8, pool=700, wide=77, page=64, least=0.3, more=16),
        # A full batch of prompts admitted and let go again, in a pool of a quarter of a million pages.
        dict(name="resize batch", op="resize", rows=512, listed=400, pool=262144, wide=1024, page=64, least=0.0, more=40000),
        # One prompt continued four ways.
        dict(name="fork one", op="fork", rows=6, sources=1, n=4, pool=200, wide=40, kv_heads=2, d=64, page=16),
        # Eight prompts continued over thirty ways each.
        dict(name="fork many", op="fork", rows=264, sources=8, n=250, pool=16384, wide=1000, kv_heads=8, d=128, page=64),
        # A small pool with holes.
        dict(name="compact small", op="compact", rows=5, pool=150, wide=33, kv_heads=2, d=64, page=16, used=0.4, common=5),
        # A large pool, a third of it in use, rows that share their first pages.
        dict(name="compact large", op="compact", rows=128, pool=16384, wide=200, kv_heads=8, d=128, page=64, used=0.33, common=50),
        # Four continuations of a short prompt, narrow heads, small pages.
        dict(name="attend few", op="attend", batch=4, groups=1, q_len=1, heads=8, kv_heads=2, d=64, page=16, least_shared=501,
             most_shared=501, most_own=40, idle=False, dtype="bf16"),
        # One decode step of a full batch behind one long document.
        dict(name="attend batch", op="attend", batch=256, groups=1, q_len=1, heads=32, kv_heads=8, d=128, page=64,
             least_shared=32768, most_shared=32768, most_own=512, idle=False, dtype="bf16"),
        # The turns of many users behind a few system prompts, taken as prompts of many tokens each; some places unused.
        dict(name="attend prompts", op="attend", batch=40, groups=3, q_len=65, heads=32, kv_heads=8, d=128, page=32,
             least_shared=2000, most_shared=9001, most_own=300, idle=True, dtype="bf16"),
        # 32-bit queries, a head of keys for each, lengths that are no multiple of anything.
        dict(name="attend fp32", op="attend", batch=13, groups=2, q_len=2, heads=16, kv_heads=16, d=80, page=32,
             least_shared=700, most_shared=3001, most_own=201, idle=False, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["copy", "resize", "fork", "compact", "attend", "attend", "attend", "attend"])
    d = 16 * rng.randint(1, 8)
    page = rng.choice([16, 32, 64, 128])
    kv_heads = _spread(rng, 1, 16)
    if op == "copy":
        room = max(8, min(20000, (1 << 31) // (kv_heads * d * page)))
        pool = _spread(rng, 8, room)
        return dict(op=op, n=_spread(rng, 1, max(1, pool * 2 // 5)), pool=pool, kv_heads=kv_heads, d=d, page=page)
    if op == "resize":
        rows, wide = _spread(rng, 1, 512), _spread(rng, 1, 1024)
        return dict(op=op, rows=rows, listed=rng.randint(1, rows), pool=rng.randint(1, rows * wide + 100) + 3, wide=wide, page=page,
                    least=rng.choice([0.0, 0.5]), more=_spread(rng, 1, max(1, wide * page // 2)))
    room = max(64, min(16384, (1 << 30) // (kv_heads * d * page)))
    if op == "fork":
        sources, wide = rng.randint(1, 8), _spread(rng, 2, 1000)
        n = _spread(rng, 1, 250)
        wide = min(wide, max(2, (room - n) // sources))
        return dict(op=op, rows=sources + n + rng.randint(0, 6), sources=sources, n=n, pool=sources * wide + n, wide=wide,
                    kv_heads=kv_heads, d=d, page=page)
    if op == "compact":
        rows, pool = _spread(rng, 1, 128), _spread(rng, 64, room)
        return dict(op=op, rows=rows, pool=pool, wide=_spread(rng, 2, 200), kv_heads=kv_heads, d=d, page=page,
                    used=rng.uniform(0.05, 0.9), common=rng.randint(0, 50))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    group, batch = rng.randint(1, 8), _spread(rng, 2, 256)
    q_len = rng.choice([1, 1, rng.randint(2, 16), _spread(rng, 17, 100)])
    # rows a head times tokens, and the bytes of what each sequence has for itself, up to those of the largest listed case
    rows = batch * q_len * group * kv_heads
    room = (1 << 28 if dtype == "bf16" else 1 << 25) // rows
    most_own = _spread(rng, q_len, max(q_len, min(2048, (1 << 27) // (batch * kv_heads * d), room // 4 + q_len)))
    most = _spread(rng, page, max(page, min(65536, room)))
    return dict(op=op, batch=batch, groups=rng.randint(1, min(8, batch)), q_len=q_len, heads=kv_heads * group, kv_heads=kv_heads, d=d,
                page=page, least_shared=rng.randint(0, most), most_shared=most, most_own=most_own, idle=rng.random() < 0.25, dtype=dtype)


# ------------------------------------------------------------------ sizes

def _even(n, lo, hi):
    """n whole numbers, evenly spaced over [lo, hi]."""
    return [lo + (hi - lo) * (i + 1) // n if n > 1 else hi for i in range(n)]


def _attend_sizes(case):
    """Of each group the first sequence and the shared tokens; of each sequence its tokens: a function of the case alone."""
    n, groups, q = case["batch"], case["groups"], case["q_len"]
    cu = [0] + [max(g, n * g * (g + 3) // (groups * (groups + 3))) for g in range(1, groups)] + [n]
    cu = [min(c, n - groups + g) for g, c in enumerate(cu)]
    shared = _even(groups, case["least_shared"], case["most_shared"])
    group_of = [g for g in range(groups) for _ in range(cu[g + 1] - cu[g])]
    own_tokens = _even(n, min(q, case["most_own"]), case["most_own"])
    # (a step that visits every place once, so that a group's lengths are mixed)
    step = next(s for s in range(n // 2 + 1, 2 * n + 2) if math.gcd(s, n) == 1)
    lengths = [shared[group_of[b]] + own_tokens[b * step % n] for b in range(n)]
    if case["idle"]:
        lengths = [0 if b % 7 == 3 else v for b, v in enumerate(lengths)]
    return cu, shared, lengths


def _fork_lengths(case):
    room = case["wide"] * case["page"]
    return _even(case["sources"], room // 2 - 3, room - 5)


def work(case):
    op = case["op"]
    if op == "attend":
        cu, shared, lengths = _attend_sizes(case)
        d, hk, page, q = case["d"], case["kv_heads"], case["page"], case["q_len"]
        alone = sum(max(0, n - shared[g]) for g in range(case["groups"]) for n in lengths[cu[g]: cu[g + 1]])
        rows = case["batch"] * q * case["heads"]
        tokens = sum(shared) + alone
        return {"bytes": 2 * tokens * hk * d + 8 * tokens * hk // page + rows * (2 * d * (2 if case["dtype"] == "bf16" else 4) + 4),
                "flops": 4 * sum(lengths) * q * case["heads"] * d}
    if op == "resize":  # the listed rows read, the pool's counts looked through, twice
        return {"bytes": 2 * (4 * case["listed"] * case["wide"] + 4 * case["pool"]), "flops": 0}
    a_page = 2 * case["kv_heads"] * (case["page"] * case["d"] + 4)
    if op == "copy":
        return {"bytes": case["n"] * (2 * a_page + 8), "flops": 0}
    if op == "fork":  # rows freed and written, pages' counts, the copies
        entries = case["n"] * case["wide"]
        return {"bytes": 8 * entries + 8 * case["pool"] + 2 * a_page * case["n"], "flops": 0}
    held = int(case["pool"] * case["used"])
    moved = held * (case["pool"] - held) // case["pool"]
    return {"bytes": 8 * case["rows"] * case["wide"] + 12 * case["pool"] + 2 * a_page * moved, "flops": 0}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _pool(g, s, pool, heads, page, d):
    """Codes and scales of `pool` pages of keys and of values, as writes left them: normal values whose size differs from page to page."""
    for name in ("k", "v"):
        codes = torch.empty(pool, heads, page, d, dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty(pool, heads, device="cuda")
        at_once = max(1, (1 << 27) // (heads * page * d))
        for first in range(0, pool, at_once):
            n = min(at_once, pool - first)
            size = torch.exp2(torch.randint(-3, 4, (n, heads, 1, 1), generator=g, device="cuda").float())
            x = torch.randn((n, heads, page, d), generator=g, device="cuda") * size
            of_page = _scale(x.abs().amax((2, 3)))
            codes[first: first + n] = (x / of_page[:, :, None, None]).to(torch.float8_e4m3fn)
            scale[first: first + n] = of_page
        s[name + "_codes"], s[name + "_scale"] = codes, scale


def _scale(amax):
    """The smallest power of two that brings `amax` to 448 or less."""
    m, e = torch.frexp(amax)
    return torch.exp2(torch.where(m <= 0.875, e - 9, e - 8).float())


def _counts(table, pool):
    """How many entries of the table hold each page."""
    return torch.bincount(table[table >= 0].long(), minlength=pool).to(torch.int32)


def _rows_of(pages, ids, wide):
    """A table whose row n holds the next pages[n] of `ids`; and how many that took."""
    n = torch.tensor(pages, device="cuda")
    table = torch.full((len(pages), wide), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(wide, device="cuda") < n[:, None]] = ids[: sum(pages)]
    return table, sum(pages)


def prepare(case, seed):
    g = _generator(seed)
    s, op, page = dict(case), case["op"], case["page"]
    if op == "copy":
        _pool(g, s, case["pool"], case["kv_heads"], page, case["d"])
        ids = _perm(g, case["pool"])
        s["src"], s["dst"] = ids[: case["n"]].contiguous(), ids[case["n"]: 2 * case["n"]].contiguous()
        return s
    if op == "resize":
        rows, wide, pool = case["rows"], case["wide"], case["pool"]
        most = wide * page - case["more"]  # (tokens before, so that `more` still fit into the row)
        before = _even(rows, int(case["least"] * max(0, most)), max(0, most))
        mine = torch.randint(0, case["more"] + 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
        before, listed_rows = _ints(before), _perm(g, rows)[: case["listed"]].contiguous()
        if case["least"] == 0.0:  # rows of no earlier tokens
            before = torch.zeros_like(before)
        # the pool's pages among the rows as far as they last; half of what is left over held elsewhere
        pages = (before + page - 1) // page
        pages = torch.where(pages.cumsum(0) <= pool, pages, torch.zeros_like(pages))
        before = torch.minimum(before, pages * page)
        ids = _perm(g, pool)
        s["table"], used = _rows_of(pages.tolist(), ids, wide)
        s["refs"] = _counts(s["table"], pool)
        s["refs"][ids[used: used + (pool - used) // 2].long()] += 1
        s["row_ids"], s["before"], s["after"] = listed_rows, before[listed_rows.long()].contiguous(), (before + mine)[listed_rows.long()].contiguous()
        return s
    if op == "fork":
        _pool(g, s, case["pool"], case["kv_heads"], page, case["d"])
        places, ids = _perm(g, case["rows"]), _perm(g, case["pool"])
        lengths = [0] * case["rows"]
        src = places[: case["sources"]].tolist()
        for place, n in zip(src, _fork_lengths(case)):
            lengths[place] = max(0, n)
        s["table"], _ = _rows_of([-(-n // page) for n in lengths], ids, case["wide"])
        s["refs"], s["lengths"] = _counts(s["table"], case["pool"]), _ints(lengths)
        s["src"] = _ints([src[i % case["sources"]] for i in range(case["n"])])
        s["dst"] = places[case["sources"]: case["sources"] + case["n"]].contiguous()
        s["none"] = torch.zeros_like(s["dst"])
        return s
    if op == "compact":
        pool, rows, wide = case["pool"], case["rows"], case["wide"]
        _pool(g, s, pool, case["kv_heads"], page, case["d"])
        held = min(int(pool * case["used"]), rows * wide)
        common = min(case["common"], wide - 1, held)
        pages = [min(wide - common, (held - common) // rows + (1 if r < (held - common) % rows else 0)) for r in range(rows)]
        ids = _perm(g, pool)
        first = ids[:common].expand(rows, common)
        rest, _ = _rows_of(pages, ids[common:], wide - common)
        s["table"] = torch.cat([first, rest], 1).contiguous()
        s["refs"] = _counts(s["table"], pool)
        s["table_to"], s["refs_to"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        return s
    cu, shared, lengths = _attend_sizes(case)
    of_prefix = [-(-n // page) for n in shared]
    wide_prefix = max(1, max(of_prefix))
    whole = [n // page for n in shared]  # pages that the group's sequences share; what else they hold is their own
    group_of = [g_ for g_ in range(case["groups"]) for _ in range(cu[g_ + 1] - cu[g_])]
    mine = [max(0, -(-n // page) - whole[group_of[b]]) for b, n in enumerate(lengths)]
    wide = max(1, max(-(-n // page) for n in lengths))
    pool = sum(of_prefix) + sum(mine) + 3
    _pool(g, s, pool, case["kv_heads"], page, case["d"])
    ids = _perm(g, pool)
    s["prefix_table"], used = _rows_of(of_prefix, ids, wide_prefix)
    own_rows, _ = _rows_of(mine, ids[used:], wide)
    at = torch.arange(wide, device="cuda")
    n_whole = torch.tensor([whole[g_] for g_ in group_of], device="cuda")[:, None]
    of_group = s["prefix_table"][torch.tensor(group_of, device="cuda")]
    table = torch.where(at < n_whole, of_group[:, at.clamp(max=wide_prefix - 1)], own_rows.gather(1, (at - n_whole).clamp(0, wide - 1)))
    need = torch.tensor([-(-n // page) for n in lengths], device="cuda")[:, None]
    s["table"] = torch.where(at < need, table, -1).to(torch.int32).contiguous()
    s["lengths"], s["prefix_lengths"], s["cu"] = _ints(lengths), _ints(shared), _ints(cu)
    s["q"] = (torch.randn((case["batch"], case["q_len"], case["heads"], case["d"]), generator=g, device="cuda") * 1.5).to(DTYPES[case["dtype"]])
    return s


# ------------------------------------------------------------------ plain forms

def _buffers(s):
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]


def _copy_plain(s, src, dst):
    src, dst = src.long(), dst.long()
    for x in _buffers(s):
        raw = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        raw[dst] = raw[src]


def _free_pages(refs):
    return torch.nonzero(refs == 0)[:, 0].to(torch.int32)


def _resize_plain(refs, table, rows, tokens, page):
    rows = rows.long()
    entries = table[rows]
    need = ((tokens + (page - 1)) // page)[:, None]
    at = torch.arange(table.shape[1], device="cuda")
    held = (entries >= 0) & (entries < len(refs))
    drop = held & (at >= need)
    refs.index_add_(0, entries[drop].long(), torch.full_like(entries[drop], -1))
    entries = torch.where(at >= need, -1, entries)
    lacks = ~held & (at < need)
    order = lacks.flatten().cumsum(0).view(lacks.shape) - 1
    free = _free_pages(refs)
    taken = lacks & (order < len(free))
    entries[taken] = free[order[taken]]
    refs[entries[taken].long()] = 1
    table[rows] = entries
    return (lacks.sum() - taken.sum()).to(torch.int32).view(1)


def _fork_plain(s):
    table, refs, lengths, page = s["table"], s["refs"], s["lengths"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    n = lengths[src]
    full = (n // page)[:, None]
    at = torch.arange(table.shape[1], device="cuda")
    entries = torch.where(at < full, table[src], -1)
    refs.index_add_(0, entries[entries >= 0].long(), torch.ones_like(entries[entries >= 0]))
    last = table[src].gather(1, full.clamp(max=table.shape[1] - 1).long())[:, 0]
    partly = (n % page > 0) & (last >= 0)
    free = _free_pages(refs)
    order = partly.cumsum(0) - 1
    taken = partly & (order < len(free))
    to = torch.full_like(last, -1)
    to[taken] = free[order[taken]]
    refs[to[taken].long()] = 1
    entries[taken, full[taken, 0].long()] = to[taken]
    table[dst] = entries
    lengths[dst] = n
    return torch.where(taken, last, -1), to, (partly.sum() - taken.sum()).to(torch.int32).view(1)


def _compact_plain(s):
    table, refs = s["table"], s["refs"]
    held = refs > 0
    n = held.sum()
    at = torch.arange(len(refs), device="cuda")
    src, dst = at[held & (at >= n)], at[~held & (at < n)]
    page_map = torch.where(held, at, -1)
    page_map[src] = dst
    refs_to = torch.where(at < n, refs, 0)
    refs_to[dst] = refs[src]
    table_to = torch.where(table >= 0, page_map[table.clamp(min=0).long()], -1)
    _copy_plain(s, src, dst)
    return table_to.to(torch.int32), refs_to, page_map.to(torch.int32), n.to(torch.int32).view(1)


def _attend_plain(s):
    """The prefix's scores by group, its rows laid side by side, then each sequence's own tokens; one softmax over both."""
    page, n_q, hk, d = s["page"], s["q_len"], s["kv_heads"], s["d"]
    group, batch, cu = s["heads"] // hk, s["batch"], s["cu"].long()
    device = s["q"].device
    shared = s["prefix_lengths"] // page * page  # whole pages: what follows them is in the sequences' own
    seq = torch.arange(batch, device=device)
    of = torch.searchsorted(cu[1:].contiguous(), seq, right=True)
    place = seq - cu[of]
    widest = place.max() + 1

    def dense(table, codes, scale):
        index = table.clamp(min=0).long()
        x = codes.view(torch.uint8)[index].view(torch.float8_e4m3fn).float() * scale[index][..., None, None]
        return x.transpose(1, 2).reshape(table.shape[0], hk, -1, d)

    q = s["q"].float().view(batch, n_q, hk, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hk, n_q * group, d)
    side = q.new_zeros(len(shared), widest, hk, n_q * group, d)
    side[of, place] = q
    side = side.transpose(1, 2).reshape(len(shared), hk, -1, d)
    mine = s["lengths"][:, None] - n_q + torch.arange(n_q, device=device, dtype=torch.int32)

    at = torch.arange(s["prefix_table"].shape[1] * page, device=device)
    k = dense(s["prefix_table"], s["k_codes"], s["k_scale"])
    before = torch.matmul(side, k.transpose(-1, -2)).view(len(shared), hk, widest, n_q * group, -1).transpose(1, 2)[of, place]
    sees = (at < shared[of][:, None])[:, None, :] & (at <= mine[:, :, None])
    before = before.view(batch, hk, n_q, group, -1).masked_fill_(~sees[:, None, :, None, :], -math.inf)

    # the sequences' own pages, from the first that they do not share on
    room = int(((s["lengths"] - shared[of]).amax().clamp(min=1) + page - 1) // page)
    first = (shared[of] // page)[:, None] + torch.arange(room, device=device, dtype=torch.int32)
    beyond = first >= s["table"].shape[1]
    table = s["table"].gather(1, first.clamp(max=s["table"].shape[1] - 1).long()).masked_fill(beyond, -1)
    at = shared[of][:, None] + torch.arange(room * page, device=device, dtype=torch.int32)
    held = (table >= 0).repeat_interleave(page, 1) & (at < s["lengths"][:, None])
    k = dense(table, s["k_codes"], s["k_scale"]).masked_fill_(~held[:, None, :, None], 0.0)
    after = torch.matmul(q, k.transpose(-1, -2)).view(batch, hk, n_q, group, -1)
    sees = held[:, None, :] & (at[:, None, :] <= mine[:, :, None])
    after = after.masked_fill_(~sees[:, None, :, None, :], -math.inf)

    score = torch.cat([before, after], -1) / math.sqrt(d)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p.view(batch, hk, n_q * group, -1)
    split = before.shape[-1]
    side = q.new_zeros(len(shared), widest, hk, n_q * group, split)
    side[of, place] = p[..., :split]
    side = side.transpose(1, 2).reshape(len(shared), hk, -1, split)
    o = torch.matmul(side, dense(s["prefix_table"], s["v_codes"], s["v_scale"]))
    o = o.view(len(shared), hk, widest, n_q * group, d).transpose(1, 2)[of, place]
    v = dense(table, s["v_codes"], s["v_scale"]).masked_fill_(~held[:, None, :, None], 0.0)
    o = o + torch.matmul(p[..., split:], v)
    o = o.view(batch, hk, n_q, group, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top)[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, n_q, s["heads"], d).to(s["q"].dtype)
    return o, lse.permute(0, 2, 1, 3).reshape(batch, n_q, s["heads"])


def run(s):
    op = s["op"]
    if own:
        import gated_delta_rule_34_gb300 as kda
        cache = kda.PagedCache(*_buffers(s)) if "k_codes" in s else None
        if op == "copy":
            kda.cache_copy(cache, s["src"], s["dst"])
            return _buffers(s)
        if op == "resize":
            kda.cache_resize(s["refs"], s["table"], s["row_ids"], s["before"], s["page"])
            missing = kda.cache_resize(s["refs"], s["table"], s["row_ids"], s["after"], s["page"])
            return s["table"], s["refs"], missing
        if op == "fork":
            kda.cache_resize(s["refs"], s["table"], s["dst"], s["none"], s["page"])
            src, dst, missing = kda.cache_fork(s["refs"], s["table"], s["lengths"], s["src"], s["dst"], s["page"])
            kda.cache_copy(cache, src, dst)
            return (s["table"], s["refs"], s["lengths"], src, dst, missing, *_buffers(s))
        if op == "compact":
            page_map, src, dst, held = kda.cache_compact(s["refs"], s["table"], refs_out=s["refs_to"], table_out=s["table_to"])
            kda.cache_copy(cache, src, dst)
            return (s["table_to"], s["refs_to"], page_map, held, *_buffers(s))
        return kda.cache_attention_shared(s["q"], cache, s["table"], s["lengths"], s["prefix_table"], s["prefix_lengths"], s["cu"],
                                          return_lse=True)
    if op == "copy":
        _copy_plain(s, s["src"], s["dst"])
        return _buffers(s)
    if op == "resize":  # the rows as they were (a step before took tokens back), then with the new tokens
        _resize_plain(s["refs"], s["table"], s["row_ids"], s["before"], s["page"])
        missing = _resize_plain(s["refs"], s["table"], s["row_ids"], s["after"], s["page"])
        return s["table"], s["refs"], missing
    if op == "fork":  # the rows of earlier forks let go, then forked
        _resize_plain(s["refs"], s["table"], s["dst"], s["none"], s["page"])
        src, dst, missing = _fork_plain(s)
        done = src >= 0
        _copy_plain(s, src[done], dst[done])
        return (s["table"], s["refs"], s["lengths"], src, dst, missing, *_buffers(s))
    if op == "compact":
        return (*_compact_plain(s), *_buffers(s))
    return _attend_plain(s)


# ------------------------------------------------------------------ from the definitions, floating ones in 64 bits

def _values(s, pairs):
    """The pool's values after copying pages, a pair after another: codes and scales as 64-bit numbers."""
    out = [x.double() for x in _buffers(s)]
    for src, dst in pairs:
        for x in out:
            x[dst] = x[src]
    return tuple(out)


def exact(case, seed):
    op, page = case["op"], case["page"]
    if op != "attend" and op != "resize" and case["pool"] * case["kv_heads"] * page * case["d"] > 1 << 31:
        return None
    s = prepare(case, seed)
    if op == "copy":
        return _values(s, zip(s["src"].tolist(), s["dst"].tolist()))
    if op in ("resize", "fork"):
        table, refs = s["table"].tolist(), s["refs"].tolist()
        if op == "resize":  # (the first call finds the rows as they are)
            free, missing = iter([p for p, n in enumerate(refs) if n == 0]), 0
            for r, n in zip(s["row_ids"].tolist(), s["after"].tolist()):
                for j in range(-(-n // page)):
                    if table[r][j] < 0:
                        table[r][j] = next(free, -1)
                        missing += table[r][j] < 0
                        if table[r][j] >= 0:
                            refs[table[r][j]] = 1
            return _ints(table), _ints(refs), _ints([missing])
        lengths, free, pairs = s["lengths"].tolist(), iter([p for p, n in enumerate(refs) if n == 0]), []
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            n = lengths[b] = lengths[a]
            for j in range(n // page):
                table[b][j] = table[a][j]
                refs[table[a][j]] += 1
            pairs.append((-1, -1))
            if n % page:
                table[b][n // page] = next(free)
                refs[table[b][n // page]] = 1
                pairs[-1] = (table[a][n // page], table[b][n // page])
        done = [p for p in pairs if p[0] >= 0]
        return (_ints(table), _ints(refs), _ints(lengths), _ints([p[0] for p in pairs]), _ints([p[1] for p in pairs]), _ints([0]), *_values(s, done))
    if op == "compact":
        refs, table = s["refs"].tolist(), s["table"].tolist()
        n = sum(r > 0 for r in refs)
        holes, late = [p for p in range(n) if refs[p] == 0], [p for p in range(n, len(refs)) if refs[p] > 0]
        page_map = [p if r > 0 else -1 for p, r in enumerate(refs)]
        for a, b in zip(late, holes):
            page_map[a], refs[b], refs[a] = b, refs[a], 0
        return (_ints([[page_map[p] if p >= 0 else -1 for p in row] for row in table]), _ints(refs), _ints(page_map), _ints([n]),
                *_values(s, zip(late, holes)))
    # attention, one sequence at a time over all of its own row, weights by the log of their sum
    n_q, hk, d = case["q_len"], case["kv_heads"], case["d"]
    group = case["heads"] // hk
    if work(case)["flops"] > 4e12:
        return None
    o = torch.zeros(case["batch"], n_q, case["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], n_q, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lengths"].tolist()):
        if not length:
            continue
        at = torch.arange(length, device="cuda")
        ids = s["table"][b].long()[at // page]
        k, v = (s[n + "_codes"].view(torch.uint8)[ids, :, at % page].view(torch.float8_e4m3fn).double() *
                s[n + "_scale"].double()[ids][..., None] for n in ("k", "v"))
        unseen = at > length - n_q + torch.arange(n_q, device="cuda")[:, None]
        for h in range(hk):
            score = torch.matmul(s["q"][b, :, h * group: (h + 1) * group].double().reshape(n_q * group, d), k[:, h].T) / math.sqrt(d)
            score = score.view(n_q, group, length).masked_fill_(unseen[:, None], -math.inf)
            total = torch.logsumexp(score, -1, keepdim=True)
            weight = torch.exp(score - torch.where(total == -math.inf, torch.zeros_like(total), total))
            o[b, :, h * group: (h + 1) * group] = torch.matmul(weight.view(n_q * group, length), v[:, h]).view(n_q, group, d)
            lse[b, :, h * group: (h + 1) * group] = total[..., 0]
    return o, lse
