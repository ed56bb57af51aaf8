"""Shared prefixes whose pages differ in size: scores far above the first ones on pages of very small values."""
import math

import pytest
import torch

from .test_gpu_cache_shared import WIDE, WIDE32, Case, both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [WIDE, WIDE32])
@pytest.mark.parametrize("n", [2, 70])                     # few rows a group, and many
@pytest.mark.parametrize("first, later", [(30, -100), (100, -100), (-100, 100)])
@pytest.mark.parametrize("size", [8.0, 32.0])
def test_scores_far_above_on_pages_of_small_values(dtype, n, first, later, size):
    """Values of 2^first in the first tile of 128 tokens, of 2^later behind it, where scores reach 2^80 to 2^400 times the weights
    before: what a row weighs against is its largest score, however little its page's values come to."""
    case = Case(25, 1, 4, 2, 64, 16, dtype, [(16 * 48, [1 + i % 40 for i in range(n)])])
    pages = case.prefix_table[0, :48].long()
    case.pool.v_scale[pages] = torch.exp2(torch.tensor([first] * 8 + [later] * 40, device="cuda").float())[:, None]
    case.pool.k_scale[pages] = torch.tensor([2.0 ** -4] * 8 + [size] * 40, device="cuda")[:, None]
    both(case)


@pytest.mark.parametrize("dtype", [WIDE, WIDE32])
@pytest.mark.parametrize("first, later", [(30, -100), (100, -100), (20, -60)])
@pytest.mark.parametrize("least, more", [(60, 1.0), (125, 0.25), (180, 1.0)])
def test_every_distance_of_scores(dtype, first, later, least, more):
    """As above, row after row a bit further, from 2^least times the weights of the first tile on."""
    case = Case(26, 1, 4, 2, 64, 16, dtype, [(16 * 48, [1 + i % 40 for i in range(70)])], spread=0)
    pages = case.prefix_table[0, :48].long()
    case.pool.k.view(torch.uint8)[pages] = 0x38            # ones
    case.pool.v_scale[pages] = torch.exp2(torch.tensor([first] * 8 + [later] * 40, device="cuda").float())[:, None]
    case.pool.k_scale[pages] = torch.tensor([2.0 ** -6] * 8 + [1.0] * 40, device="cuda")[:, None]
    far = least + more * torch.arange(70, device="cuda")[:, None, None, None] + torch.arange(4, device="cuda")[:, None] / 8
    case.q.copy_((far * math.log(2) / 8).expand_as(case.q))   # scores: 64 of them times 1, over sqrt(64)
    both(case)
