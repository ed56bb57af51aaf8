"""The example stack: a prompt and then single tokens give what one longer prompt gives."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_stack.py")


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_stack", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [dict(), dict(window=48, sinks=4), dict(scaling="by_parts", factor=4.0)])
def test_tokens_continue_a_prompt(kw):
    m = _example()
    lens, more = [70, 1, 133], 6
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = [torch.randn(1, n + more, 512, generator=gen, device="cuda").to(torch.bfloat16) for n in lens]
    whole = m.Stack(3, 160, **kw)
    want = whole.prompt(torch.cat(x, 1), [n + more for n in lens])
    stack = m.Stack(3, 160, **kw)
    first = stack.prompt(torch.cat([t[:, :n] for t, n in zip(x, lens)], 1), lens)
    steps = [stack.token(torch.cat([t[:, n + i: n + i + 1] for t, n in zip(x, lens)])) for i in range(more)]
    assert stack.lengths.tolist() == whole.lengths.tolist() == [n + more for n in lens]
    # Layers of both runs see the same values up to bf16 roundings: the recurrent prompt is a chunked
    # product in bf16 (2e-2 of the largest output is its stated bound) where single tokens are fp32, and a key whose
    # rounding to e4m3 falls the other way moves by a step of 2^-3 of itself, one key among many.
    at = 0
    for b, n in enumerate(lens):
        w = want[0, at: at + n + more].float()
        got = torch.cat([first[0, sum(lens[:b]): sum(lens[: b + 1])], torch.stack([s[b, 0] for s in steps])]).float()
        assert float((got - w).abs().max()) <= 5e-2 * float(w.abs().max()), b
        assert float((got - w).norm()) <= 1e-2 * float(w.norm()), b
        at += n + more
