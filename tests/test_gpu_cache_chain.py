"""The global-attention operators one after another without a pause: each sees all that the kernel before it wrote, whatever
that kernel is, eagerly and in a captured graph.  The same steps with a pause after each give the expected bits."""
import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu

STEPS = 12


class _Decode:
    """Decode steps, each a chain: new q, k, v from the last output, turned, written, attended to, read back."""

    def __init__(self, B, H, group, d, page, start, dtype):
        torch.manual_seed(11)
        self.B, self.dtype = B, dtype
        wide = (start + STEPS + page - 1) // page
        self.pool = kda.cache_new(B * wide, H, page, d)
        self.table = torch.randperm(B * wide, device="cuda").to(torch.int32).view(B, wide)
        if start:
            k = torch.randn(B, start, H, d, device="cuda").to(dtype)
            kda.cache_write(self.pool, k, k, self.table, torch.zeros(B, dtype=torch.int32, device="cuda"))
        self.at = torch.full((B,), start, dtype=torch.int32, device="cuda")
        self.x = torch.randn(B, 1, H * group, d, device="cuda").to(dtype)
        self.heads = H
        self.freq = kda.rotary_frequencies(d)
        self.seen = []

    def step(self, pause):
        q, k = kda.rotary(self.x, self.x[:, :, :self.heads], self.at, self.freq)
        pause()
        kda.cache_write(self.pool, k, self.x[:, :, -self.heads:], self.table, self.at)
        pause()
        lengths = self.at + 1                              # (a kernel of torch's between ours)
        o, lse = kda.cache_attention(q, self.pool, self.table, lengths, return_lse=True)
        pause()
        back, _ = kda.cache_read(self.pool, self.table, self.at, 1, dtype=self.dtype)
        pause()
        two, _ = kda.rotary(o, back, self.at, self.freq, layout="interleaved")
        pause()
        self.x.copy_(two + o)
        self.at.add_(1)
        return o, lse, back


CASES = [(1, 2, 4, 64, 16, 60, torch.bfloat16), (3, 4, 1, 128, 64, 5000, torch.float32),
         (64, 8, 4, 128, 64, 200, torch.bfloat16), (4, 2, 24, 128, 32, 3000, torch.bfloat16), (2, 2, 2, 64, 16, 0, torch.float32)]


def _run(case, pause):
    chain = _Decode(*case)
    got = [chain.step(pause) for _ in range(STEPS)]
    torch.cuda.synchronize()
    return [t.clone() for outs in got for t in outs] + [chain.x, chain.at, chain.pool.k_scale, chain.pool.k.view(torch.uint8)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_steps_without_a_pause(case):
    want = _run(case, torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(_run(case, lambda: None), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_steps_in_a_graph(case):
    want = _run(case, torch.cuda.synchronize)
    warm = _Decode(*case)
    warm.step(lambda: None)
    torch.cuda.synchronize()
    chain = _Decode(*case)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain.step(lambda: None)
    got = []
    for _ in range(STEPS):
        graph.replay()
        got += [t.clone() for t in outs]
    torch.cuda.synchronize()
    got += [chain.x, chain.at, chain.pool.k_scale, chain.pool.k.view(torch.uint8)]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_after_what_is_no_kernel():
    """After a copy, a fill and an event of another stream, eagerly and captured."""
    torch.manual_seed(12)
    x = torch.randn(8, 4, 4, 64, device="cuda")
    pos, freq = torch.arange(32, dtype=torch.int32, device="cuda"), kda.rotary_frequencies(64)
    want, _ = kda.rotary(x, None, pos, freq)
    zero = torch.zeros_like(x)
    torch.cuda.synchronize()

    def chain():
        main, side = torch.cuda.current_stream(), torch.cuda.Stream()
        y = torch.empty_like(x)
        y.copy_(x)
        a, _ = kda.rotary(y, None, pos, freq)
        y.zero_()
        b, _ = kda.rotary(y, None, pos, freq)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z = x.clone()
            c, _ = kda.rotary(z, None, pos, freq)
        main.wait_stream(side)
        d, _ = kda.rotary(z, None, pos, freq, q_out=torch.empty_like(z))
        return a, b, c, d, z

    for _ in range(5):
        a, b, c, d, _ = chain()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, zero) and torch.equal(c, want) and torch.equal(d, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b, c, d, _ = chain()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, zero) and torch.equal(c, want) and torch.equal(d, want)
