"""Plain 64-bit forms of the global-attention operators, one token at a time where it matters,
for the tests.  CPU tensors; none of the library's code."""
import math

import torch

F64 = torch.float64


def rotary(x, positions, freq, layout, amplitude):
    """x [n, H, d]; in 64 bits."""
    x = x.double().clone()
    a = positions.double()[:, None] * freq.double()
    c, s = (torch.cos(a) * amplitude)[:, None], (torch.sin(a) * amplitude)[:, None]
    r = 2 * freq.numel()
    one, two = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    u, v = x[..., one].clone(), x[..., two].clone()
    x[..., one], x[..., two] = u * c - v * s, v * c + u * s
    return x


def to_e4m3(x):
    """The nearest e4m3 value (ties to even) of each 64-bit x; beyond 448: 448; NaN: NaN."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def scale_of(values):
    """The least power of two from 2^-100 up that brings every finite value to 448 or less."""
    finite = values[torch.isfinite(values)].abs()
    amax = float(finite.max()) if finite.numel() else 0.0
    e = -100
    if amax > 0:
        e = max(e, math.frexp(amax / 448.0)[1] - 2)
        while amax > 448.0 * 2.0 ** e:
            e += 1
    return 2.0 ** e


class Cache:
    """The pool in 64 bits: the values that the codes stand for, before their scale."""

    def __init__(self, pool):
        self.codes = {n: getattr(pool, n).cpu().float().double() for n in "kv"}
        self.scale = {n: getattr(pool, n + "_scale").cpu().double() for n in "kv"}
        self.n_pages, self.heads, self.page, self.d = self.codes["k"].shape

    def page_of(self, table, n, position):
        i = position // self.page
        if i >= table.shape[1]:
            return None
        p = int(table[n, i])
        return p if 0 <= p < self.n_pages else None

    def write(self, name, rows, table, n, start):
        """rows [T, H, d]: sequence n's tokens from position start on."""
        rows, at, end = rows.cpu().double(), start, start + rows.shape[0]
        while at < end:
            upto, slot = min(end, (at // self.page + 1) * self.page), at % self.page
            p = self.page_of(table, n, at)
            if p is not None:
                part = rows[at - start: upto - start]
                for h in range(self.heads):
                    s, old = scale_of(part[:, h]), float(self.scale[name][p, h])
                    if slot and old > s:
                        s = old
                    if slot and s > old:
                        self.codes[name][p, h, :slot] = to_e4m3(self.codes[name][p, h, :slot] * (old / s))
                    self.codes[name][p, h, slot: slot + upto - at] = to_e4m3(part[:, h] / s)
                    self.scale[name][p, h] = s
            at = upto

    def values(self, name, table, n, position):
        """[H, d] of one token, or None where its page is not held."""
        p = self.page_of(table, n, position)
        if p is None:
            return None
        return self.codes[name][p, :, position % self.page] * self.scale[name][p][:, None]


def attention(q, cache, table, lengths, scale, window=0, sinks=0):
    """o, lse, and what bounds a row's error: sum of w |v|, the largest sum of |q k| scale, and the largest w times
    its page's scale of v, times the sum of |v| / scale.  64 bits."""
    q = q.cpu().double()
    B, t_q, h_q, d = q.shape
    group = h_q // cache.heads
    o, weight = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    lse = torch.full((B, t_q, h_q), -math.inf, dtype=F64)
    size = torch.zeros((B, t_q, h_q), dtype=F64)
    floor = torch.zeros(q.shape, dtype=F64)
    for b in range(B):
        length = max(0, min(int(lengths[b]), table.shape[1] * cache.page))
        if length == 0:
            continue
        got = [(t, cache.values("k", table, b, t), cache.values("v", table, b, t)) for t in range(length)]
        got = [g for g in got if g[1] is not None]
        if not got:
            continue
        at = torch.tensor([g[0] for g in got])
        k, v = torch.stack([g[1] for g in got]), torch.stack([g[2] for g in got])   # [t, H_kv, d]
        of_page = torch.stack([cache.scale["v"][cache.page_of(table, b, g[0])] for g in got])   # [t, H_kv]
        for i in range(t_q):
            p = length - t_q + i
            sees = at <= p
            if window:
                sees &= (at > p - window) | (at < sinks)
            if not bool(sees.any()):
                continue
            for h in range(h_q):
                kk, vv = k[sees, h // group], v[sees, h // group]
                s = scale * (kk * q[b, i, h]).sum(-1)
                m = s.max()
                if m == -math.inf:
                    continue
                lse[b, i, h] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[b, i, h])
                o[b, i, h] = (w[:, None] * vv).sum(0)
                weight[b, i, h] = (w[:, None] * vv.abs()).sum(0)
                vs = of_page[sees, h // group]
                floor[b, i, h] = (w * vs).max() * (vv.abs() / vs[:, None]).sum(0)
                size[b, i, h] = abs(scale) * (kk * q[b, i, h]).abs().sum(-1).max()
    return o, lse, weight, size, floor
