"""Cases for measuring the serving operators of a global-attention layer beside the recurrent layers.

Four operators, in plain torch (``own`` false) or through this package (``own`` true):

  rotary   rotary positions on a step's queries and keys
  write    new keys and values quantised to e4m3 as they enter a paged cache, with one power-of-two
           scale for each page and head
  read     the cached tokens of some positions, back as dense rows
  attend   attention of the newest tokens of each sequence over that cache

A case is a dict of plain values; every random number comes from the seed.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_NAN = 0x7F
SCALE_MIN_EXP = -100


def listed():
    return [
        # One sequence's next token: two small rows, so launch latency is everything.
        dict(name="rotary one token", op="rotary", tokens=1, heads=16, kv_heads=4, d=128, rot=128, layout="half",
             dtype="bf16", base=10000.0, scaling="none", factor=1.0, trained=8192, far=32768, fused=True),
        # A long prompt of a wide layer, half of each head rotated, positions far beyond the trained length.
        dict(name="rotary prompt", op="rotary", tokens=65536, heads=32, kv_heads=8, d=128, rot=64, layout="interleaved",
             dtype="bf16", base=500000.0, scaling="by_parts", factor=16.0, trained=65536, far=1048576, fused=True),
        # An odd number of tokens in 32 bits, narrow heads, as in a reference run.
        dict(name="rotary fp32", op="rotary", tokens=4097, heads=16, kv_heads=16, d=64, rot=64, layout="half",
             dtype="f32", base=10000.0, scaling="linear", factor=4.0, trained=4096, far=16384, fused=False),
        # One decode step of a full batch: a token for each sequence into a page that is partly filled.
        dict(name="write one token each", op="write", batch=256, min_new=1, max_new=1, kv_heads=8, d=128, page=64,
             max_start=1024, dtype="bf16", fused=True),
        # Prompts of unequal lengths packed one after another, some continuing earlier turns.
        dict(name="write packed prompts", op="write", batch=64, min_new=1, max_new=4096, kv_heads=16, d=128, page=64,
             max_start=1000, dtype="bf16", fused=True),
        # A prefix brought back as dense rows, to go on with it elsewhere.
        dict(name="read prefix", op="read", batch=16, min_len=1, max_len=16384, kv_heads=8, d=128, page=64,
             max_start=100, dtype="bf16"),
        # The first turns of one short chat: a few dozen tokens, narrow heads, small pages.
        dict(name="attend short", op="attend", batch=1, q_len=1, heads=8, kv_heads=2, d=64, page=16, min_len=77,
             max_len=77, window=0, sinks=0, dropped=False, dtype="bf16"),
        # One decode step of a full batch with lengths all over the range.
        dict(name="attend batch", op="attend", batch=256, q_len=1, heads=32, kv_heads=8, d=128, page=64, min_len=1,
             max_len=4096, window=0, sinks=0, dropped=False, dtype="bf16"),
        # One sequence of a million tokens: all of the GPU on a single token.
        dict(name="attend million", op="attend", batch=1, q_len=1, heads=32, kv_heads=8, d=128, page=64,
             min_len=1048576, max_len=1048576, window=0, sinks=0, dropped=False, dtype="bf16"),
        # Draft tokens of speculative decoding, verified together.
        dict(name="attend drafts", op="attend", batch=32, q_len=8, heads=32, kv_heads=8, d=128, page=64, min_len=1000,
             max_len=16384, window=0, sinks=0, dropped=False, dtype="bf16"),
        # A sliding window with the first tokens kept, the pages between them given back.
        dict(name="attend window", op="attend", batch=32, q_len=1, heads=32, kv_heads=4, d=128, page=32, min_len=100,
             max_len=32768, window=4096, sinks=4, dropped=True, dtype="bf16"),
        # 32-bit queries, a head of keys for each, lengths that are no multiple of anything.
        dict(name="attend fp32", op="attend", batch=8, q_len=3, heads=16, kv_heads=16, d=80, page=32, min_len=0,
             max_len=1501, window=0, sinks=0, dropped=False, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = 16 * rng.randint(1, 8)
    page = rng.choice([16, 32, 64, 128])
    kv_heads = _spread(rng, 1, 16)
    group = rng.randint(1, 8)
    if op == "rotary":
        heads = kv_heads * group
        room = (1 << 28) // ((heads + kv_heads) * d * (1 if dtype == "bf16" else 2))
        return dict(op=op, tokens=_spread(rng, 1, min(65536, room)), heads=heads, kv_heads=kv_heads, d=d,
                    rot=2 * rng.randint(1, d // 2), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                    base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "by_parts"]),
                    factor=rng.choice([2.0, 4.0, 16.0]), trained=_spread(rng, 4096, 65536),
                    far=_spread(rng, 4096, 16777216), fused=rng.random() < 0.5)
    if op in ("write", "read"):
        batch = _spread(rng, 1, 256)
        room = (1 << 28) // (batch * kv_heads * d * (1 if dtype == "bf16" else 2))
        most = _spread(rng, 1, max(1, min(16384, room)))
        least = rng.randint(0, most)
        if op == "write":
            return dict(op=op, batch=batch, min_new=least, max_new=most, kv_heads=kv_heads, d=d, page=page,
                        max_start=_spread(rng, 1, 1024), dtype=dtype, fused=rng.random() < 0.5)
        return dict(op=op, batch=batch, min_len=least, max_len=most, kv_heads=kv_heads, d=d, page=page,
                    max_start=_spread(rng, 1, 1000), dtype=dtype)
    batch = _spread(rng, 1, 256)
    room = (1 << 28) // (batch * kv_heads * d)
    most = _spread(rng, 1, max(1, min(262144, room)))
    window = rng.choice([0, 0, _spread(rng, 1, 8192)])
    return dict(op=op, batch=batch, q_len=rng.choice([1, 1, 1, rng.randint(2, 16)]), heads=kv_heads * group,
                kv_heads=kv_heads, d=d, page=page, min_len=rng.randint(0, most), max_len=most, window=window,
                sinks=rng.randint(0, 8) if window else 0, dropped=bool(window) and rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------------ sizes

def _lengths(case, least, most):
    """The batch's lengths, evenly spaced over [least, most]: a function of the case alone."""
    n, lo, hi = case["batch"], case[least], case[most]
    return [lo + (hi - lo) * (i + 1) // n if n > 1 else hi for i in range(n)]


def _seen(case, length):
    """How many tokens of a sequence at least one of its queries sees."""
    if not case["window"]:
        return length
    first = max(0, length - case["q_len"] - case["window"] + 1)
    return length - first + min(case["sinks"], first)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    d, hk = case["d"], case["kv_heads"]
    if case["op"] == "rotary":
        values = case["tokens"] * (case["heads"] + hk) * d
        turned = values * case["rot"] // d
        return {"bytes": 2 * values * size + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * turned}
    if case["op"] == "write":
        rows = sum(_lengths(case, "min_new", "max_new")) * hk
        return {"bytes": 2 * rows * d * (size + 1) + 8 * case["batch"] * hk, "flops": 4 * rows * d}
    if case["op"] == "read":
        rows = sum(_lengths(case, "min_len", "max_len")) * hk
        return {"bytes": 2 * rows * d * (size + 1) + 8 * case["batch"] * hk, "flops": 2 * rows * d}
    seen = sum(_seen(case, n) for n in _lengths(case, "min_len", "max_len"))
    rows = case["batch"] * case["q_len"] * case["heads"]
    return {"bytes": 2 * seen * hk * d + 8 * seen * hk // case["page"] + rows * (2 * d * size + 4),
            "flops": 4 * seen * case["q_len"] * case["heads"] * d}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t[torch.randperm(len(values), generator=g, device="cuda")]


def _table(g, tokens, page, most):
    """A block table whose rows cover `tokens` each, its pages scattered over a pool that has room for `most` each; and the pool's size."""
    pages = [-(-n // page) for n in tokens]
    wide = max(1, max(pages))
    pool = sum(-(-n // page) for n in most) + 3
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    used = torch.arange(wide, device="cuda")[None, :] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.full((len(tokens), wide), -1, dtype=torch.int32, device="cuda")
    table[used] = ids[: sum(pages)]
    return table, pool


def _pool(g, pool, heads, page, d):
    """Codes and scales of `pool` pages, as earlier writes left them: normal values whose size differs from page to page."""
    size = torch.exp2(torch.randint(-3, 4, (pool, heads, 1, 1), generator=g, device="cuda").float())
    x = _normal(g, pool, heads, page, d) * size
    scale = _scale(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _generator(seed)
    dtype, d, hk = DTYPES[case["dtype"]], case["d"], case["kv_heads"]
    s = dict(case)
    if case["op"] == "rotary":
        n, h = case["tokens"], case["heads"]
        if case["fused"]:  # views of one projection's output, the values' part included
            qkv = _normal(g, n, (h + 2 * hk) * d).to(dtype)
            s["q"] = qkv[:, : h * d].view(n, h, d)
            s["k"] = qkv[:, h * d: (h + hk) * d].view(n, hk, d)
        else:
            s["q"], s["k"] = _normal(g, n, h, d).to(dtype), _normal(g, n, hk, d).to(dtype)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
        freq = case["base"] ** (-i / case["rot"])
        if case["scaling"] == "linear":
            freq = freq / case["factor"]
        elif case["scaling"] == "by_parts":
            turns = case["trained"] * freq / (2 * math.pi)
            keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
            freq = freq * (keep + (1.0 - keep) / case["factor"])
        s["freq"] = freq
        s["amplitude"] = 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "by_parts" else 1.0
        return s
    if case["op"] == "write":
        new = _shuffled(_lengths(case, "min_new", "max_new"), g)
        start = torch.randint(0, case["max_start"] + 1, (case["batch"],), generator=g, device="cuda", dtype=torch.int32)
        s["table"], pool = _table(g, (start + new).tolist(), case["page"],
                                  [n + case["max_start"] for n in _lengths(case, "min_new", "max_new")])
        s["k_codes"], s["k_scale"] = _pool(g, pool, hk, case["page"], d)
        s["v_codes"], s["v_scale"] = _pool(g, pool, hk, case["page"], d)
        s["start"], total = start, int(new.sum())
        s["cu"] = torch.cat([new.new_zeros(1), new.cumsum(0, dtype=torch.int32)])
        if case["fused"]:
            kv = _normal(g, 1, total, 2 * hk * d, std=2.0).to(dtype)
            s["new_k"], s["new_v"] = (kv[..., i * hk * d: (i + 1) * hk * d].view(1, total, hk, d) for i in (0, 1))
        else:
            s["new_k"], s["new_v"] = (_normal(g, 1, total, hk, d, std=2.0).to(dtype) for _ in (0, 1))
        return s
    if case["op"] == "read":
        n = _shuffled(_lengths(case, "min_len", "max_len"), g)
        s["start"] = torch.randint(0, case["max_start"] + 1, (case["batch"],), generator=g, device="cuda", dtype=torch.int32)
        s["table"], pool = _table(g, (s["start"] + n).tolist(), case["page"],
                                  [n + case["max_start"] for n in _lengths(case, "min_len", "max_len")])
        s["k_codes"], s["k_scale"] = _pool(g, pool, hk, case["page"], d)
        s["v_codes"], s["v_scale"] = _pool(g, pool, hk, case["page"], d)
        s["cu"], s["total"] = torch.cat([n.new_zeros(1), n.cumsum(0, dtype=torch.int32)]), int(n.sum())
        return s
    lengths = _shuffled(_lengths(case, "min_len", "max_len"), g)
    s["lengths"], page = lengths, case["page"]
    s["table"], pool = _table(g, lengths.tolist(), page, lengths.tolist())
    s["k_codes"], s["k_scale"] = _pool(g, pool, hk, page, d)
    s["v_codes"], s["v_scale"] = _pool(g, pool, hk, page, d)
    # what lies in a page past its sequence's end is whatever was there: here, bytes that are no number
    index = torch.arange(s["table"].shape[1], device="cuda")
    filled = (lengths[:, None] - index * page).clamp(0, page)
    of_page = torch.full((pool,), 0, dtype=torch.int64, device="cuda")
    of_page[s["table"][s["table"] >= 0].long()] = filled[s["table"] >= 0].long()
    stale = (torch.arange(page, device="cuda") >= of_page[:, None])[:, None, :, None]
    for name in ("k_codes", "v_codes"):
        s[name].view(torch.uint8).masked_fill_(stale, E4M3_NAN)
    if case["dropped"]:  # pages that no query sees any more have been given back
        first = (lengths - case["q_len"] - case["window"] + 1).clamp(min=0)
        gone = (index * page >= case["sinks"]) & ((index + 1) * page <= first[:, None])
        s["table"] = torch.where(gone, torch.full_like(s["table"], -1), s["table"])
    s["q"] = _normal(g, case["batch"], case["q_len"], case["heads"], d, std=1.5).to(dtype)
    return s


# ------------------------------------------------------------------ plain forms

def _scale(amax):
    """The smallest power of two, at least 2^-100, that brings `amax` to 448 or less."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_MIN_EXP)).clamp(min=SCALE_MIN_EXP)
    return torch.exp2(e.float())


def _rotary_plain(s):
    angle = s["positions"].double()[:, None] * s["freq"]
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["amplitude"]).float()[:, None, :]
    rot = s["rot"]

    def turned(x):
        f = x.float()
        if s["layout"] == "half":
            a, b = f[..., : rot // 2], f[..., rot // 2: rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = f[..., 0:rot:2], f[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([y, f[..., rot:]], -1).to(x.dtype)

    return turned(s["q"]), turned(s["k"])


def _places(s, total):
    """Of each packed token: its sequence, page and slot."""
    t = torch.arange(total, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    at = (s["start"][seq] + t - s["cu"][seq]).long()
    return seq, s["table"][seq, at // s["page"]].long(), at % s["page"]


def _write_plain(s):
    total = s["new_k"].shape[1]
    if total:
        seq, pages, slots = _places(s, total)
        n_new = (s["cu"][1:] - s["cu"][:-1]).long()
        offset = s["start"].long() % s["page"]
        carried = (offset > 0) & (n_new > 0)  # sequences whose first touched page already holds tokens
        first = s["table"][torch.arange(len(n_new), device="cuda"), (s["start"] // s["page"]).clamp(max=s["table"].shape[1] - 1).long()].long()[carried]
        older = torch.arange(s["page"], device="cuda")[None, :] < offset[carried][:, None]
        for name in ("k", "v"):
            codes, scale, x = s[name + "_codes"], s[name + "_scale"], s["new_" + name][0].float()
            amax = torch.zeros_like(scale)
            amax.index_reduce_(0, pages, x.abs().amax(-1), "amax")
            new = torch.where(torch.zeros_like(scale).index_fill_(0, pages, 1.0) > 0, _scale(amax), scale)
            new[first] = torch.maximum(new[first], scale[first])
            kept = codes.view(torch.uint8)[first]
            moved = (kept.view(torch.float8_e4m3fn).float() * (scale[first] / new[first])[:, :, None, None]).to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[first] = torch.where(older[:, None, :, None], moved.view(torch.uint8), kept)
            rows = (x / new[pages][:, :, None]).to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[pages, :, slots] = rows.view(torch.uint8)
            scale.copy_(new)
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]


def _read_plain(s):
    _, pages, slots = _places(s, s["total"])

    def rows(codes, scale):
        x = codes.view(torch.uint8)[pages, :, slots].view(torch.float8_e4m3fn).float() * scale[pages][:, :, None]
        return x.to(DTYPES[s["dtype"]])[None]

    return rows(s["k_codes"], s["k_scale"]), rows(s["v_codes"], s["v_scale"])


def _attend_plain(s):
    table, page, n_q = s["table"], s["page"], s["q_len"]
    batch, wide = table.shape
    hk, d = s["kv_heads"], s["d"]
    group = s["heads"] // hk
    at = torch.arange(wide * page, device="cuda")
    held = (at < s["lengths"][:, None]) & (table >= 0).repeat_interleave(page, 1)
    mine = s["lengths"][:, None] - n_q + torch.arange(n_q, device="cuda")
    sees = held[:, None, :] & (at <= mine[:, :, None])
    if s["window"]:
        sees = sees & ((at < s["sinks"]) | (at > mine[:, :, None] - s["window"]))
    index = table.clamp(min=0).long()

    def dense(codes, scale):
        x = codes.view(torch.uint8)[index].view(torch.float8_e4m3fn).float() * scale[index][..., None, None]
        return x.transpose(1, 2).reshape(batch, hk, wide * page, d).masked_fill(~held[:, None, :, None], 0.0)

    q = s["q"].float().view(batch, n_q, hk, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hk, n_q * group, d)
    score = torch.matmul(q, dense(s["k_codes"], s["k_scale"]).transpose(-1, -2)) / math.sqrt(d)
    score = score.view(batch, hk, n_q, group, -1).masked_fill(~sees[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, hk, n_q * group, -1), dense(s["v_codes"], s["v_scale"]))
    o = o.view(batch, hk, n_q, group, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top)[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, n_q, s["heads"], d).to(s["q"].dtype)
    return o, lse.permute(0, 2, 1, 3).reshape(batch, n_q, s["heads"])


def run(s):
    if own:
        import gated_delta_rule_34_gb300 as kda
        if s["op"] == "rotary":
            return kda.rotary(s["q"], s["k"], s["positions"], s["freq"], layout=s["layout"], amplitude=s["amplitude"])
        cache = kda.PagedCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        if s["op"] == "write":
            kda.cache_write(cache, s["new_k"], s["new_v"], s["table"], s["start"], cu_seqlens=s["cu"])
            return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
        if s["op"] == "read":
            return kda.cache_read(cache, s["table"], s["start"], s["total"], cu_seqlens=s["cu"], dtype=DTYPES[s["dtype"]])
        return kda.cache_attention(s["q"], cache, s["table"], s["lengths"], window=s["window"], sinks=s["sinks"],
                                   return_lse=True)
    return {"rotary": _rotary_plain, "write": _write_plain, "read": _read_plain, "attend": _attend_plain}[s["op"]](s)


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _to_e4m3(x):
    """64-bit values rounded to the nearest value of e4m3 (ties to even): 3 bits of fraction, least exponent -6."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(exponent - 3.0)
    return torch.round(x / step) * step


def _exact_scale(amax):
    """The power-of-two scale of blocks, from the definition: the least exponent from -100 up whose 448 is no less."""
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -130))) - 10.0
    for _ in range(3):
        e = torch.where(amax > 448.0 * torch.exp2(e), e + 1.0, e)
    return torch.exp2(e.clamp(min=float(SCALE_MIN_EXP)))


def exact(case, seed):
    if case["op"] == "write" and sum(_lengths(case, "min_new", "max_new")) * case["kv_heads"] > 3_000_000:
        return None
    s = prepare(case, seed)
    if case["op"] == "rotary":
        z = torch.exp(1j * (s["positions"].double()[:, None] * s["freq"])) * s["amplitude"]
        out = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            r = case["rot"]
            first, second = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
            w = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z[:, None, :]
            y[..., first], y[..., second] = w.real, w.imag
            out.append(y)
        return tuple(out)
    page, table = case["page"], s["table"].tolist()
    if case["op"] == "write":
        # A page at a time, over all heads: the block's scale, the older tokens moved to it, the new ones rounded.
        start, cu, done = s["start"].tolist(), s["cu"].tolist(), []
        for name in ("k", "v"):
            values, scale = s[name + "_codes"].double(), s[name + "_scale"].double()
            x = s["new_" + name][0].double()
            for b in range(case["batch"]):
                at, end = start[b], start[b] + cu[b + 1] - cu[b]
                while at < end:
                    upto, at_page, slot = min(end, (at // page + 1) * page), table[b][at // page], at % page
                    rows = x[cu[b] + at - start[b]: cu[b] + upto - start[b]].transpose(0, 1)
                    new = _exact_scale(rows.abs().amax((1, 2)))
                    if slot:
                        new = torch.maximum(new, scale[at_page])
                        values[at_page, :, :slot] = _to_e4m3(values[at_page, :, :slot] * (scale[at_page] / new)[:, None, None])
                    values[at_page, :, slot: slot + upto - at] = _to_e4m3(rows / new[:, None, None])
                    scale[at_page] = new
                    at = upto
            done.append((values, scale))
        return done[0][0], done[1][0], done[0][1], done[1][1]
    if case["op"] == "read":
        start, cu, out = s["start"].tolist(), s["cu"].tolist(), []
        for name in ("k", "v"):
            rows = []
            for b in range(case["batch"]):
                n = cu[b + 1] - cu[b]
                if not n:
                    continue
                first, last = start[b] // page, (start[b] + n - 1) // page
                ids = torch.tensor(table[b][first: last + 1], device="cuda")
                x = s[name + "_codes"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * s[name + "_scale"][ids].double()[:, :, None, None]
                rows.append(x.permute(0, 2, 1, 3).flatten(0, 1)[start[b] - first * page:][:n])
            out.append(torch.cat(rows)[None] if rows else torch.zeros(1, 0, case["kv_heads"], case["d"], dtype=torch.float64, device="cuda"))
        return tuple(out)
    # attention, one sequence at a time: gathered visible tokens, weights by the log of their sum
    n_q, hk, group, d = case["q_len"], case["kv_heads"], case["heads"] // case["kv_heads"], case["d"]
    o = torch.zeros(case["batch"], n_q, case["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], n_q, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lengths"].tolist()):
        for i in range(n_q):
            p = length - n_q + i
            if p < 0:
                continue
            at = torch.arange(p + 1, device="cuda")
            if case["window"]:
                at = at[(at < case["sinks"]) | (at > p - case["window"])]
            ids = s["table"][b].long()[at // page]
            at, ids = at[ids >= 0], ids[ids >= 0]
            if not at.numel():
                continue
            k, v = (s[n + "_codes"].view(torch.uint8)[ids, :, at % page].view(torch.float8_e4m3fn).double() *
                    s[n + "_scale"].double()[ids][..., None] for n in ("k", "v"))
            score = torch.einsum("hgd,thd->hgt", s["q"][b, i].double().view(hk, group, d), k) / math.sqrt(d)
            total = torch.logsumexp(score, -1)
            o[b, i] = torch.einsum("hgt,thd->hgd", torch.exp(score - total[..., None]), v).reshape(-1, d)
            lse[b, i] = total.reshape(-1)
    return o, lse
