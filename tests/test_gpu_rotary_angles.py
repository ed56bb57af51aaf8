"""Rotary angles to the last bits: with (1, 0) turned, the outputs are cos and sin themselves.

The bound.  The angle is off by 2^-32 turns of its fixed point and p 2^-53 turns of the frequency's product; cos and sin are
within 2 steps of their last place of the rounded ones of that angle (a step is at most 2^-23 of the value), here 2^-21.5 of it to
allow for the steps of a corrected angle.  So where sin or cos is small, near whole and half turns and quarters between them, it
must still have its digits.
"""
import math

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu


def _turned(position, freq, layout):
    x = torch.zeros(len(position), 1, 8, device="cuda")
    x[..., 0] = 1.0
    y, _ = kda.rotary(x, None, position.to(torch.int32).cuda(), freq.cuda(), layout=layout)
    return y[:, 0, 0].double().cpu(), y[:, 0, 1 if layout == "interleaved" else 4].double().cpu()


def _check(position, freq, layout):
    cos, sin = _turned(position, freq, layout)
    angle = position.double() * freq[0]
    turns = 2.0 ** -32 + position.double().abs() * 2.0 ** -53 * max(1.0, float(freq[0].abs()))
    for got, want in ((cos, torch.cos(angle)), (sin, torch.sin(angle))):
        tol = 2 * math.pi * turns + 2.0 ** -21.5 * want.abs()
        err = (got - want).abs()
        assert bool((err <= tol).all()), (float((err / tol).max()), int(position[(err / tol).argmax()]))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rate", [1.0, 0.1, 1e-4, 0.731])
def test_cos_and_sin(layout, rate):
    g = torch.Generator().manual_seed(7)
    freq = torch.tensor([rate, 0.5, 0.25, 0.125], dtype=torch.float64)
    position = torch.cat([torch.arange(0, 3000), torch.randint(-(1 << 20), 1 << 20, (60_000,), generator=g)])
    _check(position, freq, layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_near_quarter_turns(layout):
    """Positions beside every quarter of a turn, at 2^-12 of a turn a position: angles of 2^-12 turns and less from it."""
    for rate in (2 * math.pi * 2.0 ** -12, 2 * math.pi * (2.0 ** -2 + 2.0 ** -20), 2 * math.pi * (0.5 - 2.0 ** -22)):
        freq = torch.tensor([rate, 0.5, 0.25, 0.125], dtype=torch.float64)
        _check(torch.arange(-9000, 9000), freq, layout)


def test_quarter_turns_themselves():
    """At an eighth of a turn a position, as nearly as 64 bits hold it."""
    freq = torch.tensor([math.pi / 4, 0.5, 0.25, 0.125], dtype=torch.float64)
    cos, sin = _turned(torch.arange(0, 4096), freq, "half")
    r = 0.7071067811865476
    want = torch.tensor([1.0, r, 0.0, -r, -1.0, -r, 0.0, r], dtype=torch.float64)
    i = torch.arange(0, 4096)
    assert float((cos - want[i % 8]).abs().max()) <= 2.0 ** -23 and float((sin - want[(i + 6) % 8]).abs().max()) <= 2.0 ** -23
