"""A small hybrid stack served with this library: three recurrent layers to one of global attention.

    python examples/hybrid_stack.py [--layers 4] [--prompt 1000] [--new 32]

Random weights, no vocabulary: hidden states go in and come out.  A prompt of several sequences of
unequal lengths is taken at once (packed), then one token a step.  Each recurrent layer keeps
a fixed fp32 state a sequence (chunk_prefill, decode_step); each global layer turns its queries and
keys by their positions (rotary), puts keys and values into its paged 8-bit cache (cache_write) and
attends over it (cache_attention).  The projections around them are plain matrix products.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_delta_rule_34_gb300 as kda  # noqa: E402

D, PAGE = 128, 64


def _norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def _unit(x):
    return (x.float() / x.float().norm(dim=-1, keepdim=True).clamp_min(1e-30)).to(x.dtype)


class RecurrentLayer:
    """Kimi Delta Attention with its projections; the state is [N, H, D, D] fp32."""

    def __init__(self, width, heads, n_seqs, gen):
        self.heads = heads
        self.w_in = torch.randn(width, heads * (4 * D + 1), generator=gen, device="cuda").to(torch.bfloat16) / width ** 0.5
        self.w_out = torch.randn(heads * D, width, generator=gen, device="cuda").to(torch.bfloat16) / (heads * D) ** 0.5
        self.A = torch.randn(heads, D, generator=gen, device="cuda") * 0.5
        self.state = torch.zeros(n_seqs, heads, D, D, device="cuda")

    def _inputs(self, x):
        y = _norm(x) @ self.w_in
        q, k, v, z = (y[..., i * self.heads * D: (i + 1) * self.heads * D].unflatten(-1, (self.heads, D)) for i in range(4))
        beta = torch.sigmoid(y[..., 4 * self.heads * D:].float()).to(x.dtype)
        return [t.contiguous() for t in (_unit(q), _unit(k), v, z)] + [beta.contiguous()]

    def prompt(self, x, cu):
        o, self.state = kda.chunk_prefill(*self._inputs(x), self.A, initial_state=self.state, cu_seqlens=cu)
        return x + o.flatten(-2) @ self.w_out

    def token(self, x):
        o = kda.decode_step(*(t[:, 0].contiguous() for t in self._inputs(x)), self.A, self.state)
        return x + o.flatten(-2)[:, None] @ self.w_out


class GlobalLayer:
    """Attention over everything before (or a window of it), through a paged 8-bit cache."""

    def __init__(self, width, heads, kv_heads, table, n_pages, freq, gen, window=0, sinks=0):
        self.heads, self.kv_heads, self.table, self.freq = heads, kv_heads, table, freq
        self.window, self.sinks = window, sinks
        self.w_in = torch.randn(width, (heads + 2 * kv_heads) * D, generator=gen, device="cuda").to(torch.bfloat16) / width ** 0.5
        self.w_out = torch.randn(heads * D, width, generator=gen, device="cuda").to(torch.bfloat16) / (heads * D) ** 0.5
        self.cache = kda.cache_new(n_pages, kv_heads, PAGE, D)

    def _qkv(self, x, positions):
        y = _norm(x) @ self.w_in                          # views of one projection: strided, not copied
        q, k, v = (y[..., a * D: b * D].unflatten(-1, (b - a, D)) for a, b in
                   ((0, self.heads), (self.heads, self.heads + self.kv_heads),
                    (self.heads + self.kv_heads, self.heads + 2 * self.kv_heads)))
        kda.rotary(q, k, positions, self.freq, q_out=q, k_out=k)
        return q, k, v

    def prompt(self, x, cu, start, lengths):
        """x [1, T, width]: the sequences' new tokens packed, sequence n's from position start[n] on."""
        new = lengths - start
        seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), new.long())
        positions = (torch.arange(x.shape[1], device="cuda", dtype=torch.int32) - cu[seq] + start[seq]).to(torch.int32)
        q, k, v = self._qkv(x, positions)
        kda.cache_write(self.cache, k, v, self.table, start, cu_seqlens=cu)
        out = torch.empty(1, x.shape[1], self.heads, D, dtype=x.dtype, device="cuda")
        ends = cu.tolist()
        for n in range(len(lengths)):                     # the newest tokens of one sequence a call
            if ends[n + 1] > ends[n]:
                kda.cache_attention(q[:, ends[n]: ends[n + 1]], self.cache, self.table[n: n + 1], lengths[n: n + 1],
                                    window=self.window, sinks=self.sinks, out=out[:, ends[n]: ends[n + 1]])
        return x + out.flatten(-2) @ self.w_out

    def token(self, x, position):
        """x [N, 1, width], one token of every sequence, at position[n]."""
        q, k, v = self._qkv(x, position[:, None].contiguous())
        kda.cache_write(self.cache, k, v, self.table, position)
        o = kda.cache_attention(q, self.cache, self.table, position + 1, window=self.window, sinks=self.sinks)
        return x + o.flatten(-2) @ self.w_out


class Stack:
    def __init__(self, n_seqs, room, width=512, heads=4, kv_heads=2, layers=4, seed=0, window=0, sinks=0, scaling="none",
                 factor=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        pages = -(-room // PAGE)
        table = torch.randperm(n_seqs * pages, generator=gen, device="cuda").to(torch.int32).view(n_seqs, pages)
        freq = kda.rotary_frequencies(D, scaling=scaling, factor=factor, trained_len=4096)
        self.lengths = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.layers = [GlobalLayer(width, heads, kv_heads, table, n_seqs * pages, freq, gen, window, sinks) if i % 4 == 3
                       else RecurrentLayer(width, heads, n_seqs, gen) for i in range(layers)]

    def prompt(self, x, lens):
        """x [1, sum(lens), width], the sequences' next tokens one after another."""
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = torch.cat([new.new_zeros(1), new.cumsum(0, dtype=torch.int32)])
        start, self.lengths = self.lengths, self.lengths + new
        for layer in self.layers:
            x = layer.prompt(x, cu, start, self.lengths) if isinstance(layer, GlobalLayer) else layer.prompt(x, cu)
        return x

    def token(self, x):
        """x [N, 1, width], the next token of every sequence."""
        position, self.lengths = self.lengths, self.lengths + 1
        for layer in self.layers:
            x = layer.token(x, position) if isinstance(layer, GlobalLayer) else layer.token(x)
        return x


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--new", type=int, default=32)
    a = ap.parse_args()
    lens = [a.prompt, max(1, a.prompt // 3), 1, max(1, a.prompt // 2 + 7)]
    stack = Stack(len(lens), a.prompt + a.new, layers=a.layers)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, sum(lens), 512, generator=gen, device="cuda").to(torch.bfloat16)
    y = stack.prompt(x, lens)
    ends = torch.tensor(lens).cumsum(0) - 1
    x = y[0, ends.cuda()][:, None]
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.new):
        x = _norm(stack.token(x))
    end.record()
    torch.cuda.synchronize()
    print(f"{sum(lens)} prompt tokens of {len(lens)} sequences, then {a.new} steps of {len(lens)} tokens: "
          f"{start.elapsed_time(end) / max(1, a.new):.3f} ms a step, lengths {stack.lengths.tolist()}")


if __name__ == "__main__":
    main()
