"""Attention under windows that no sequence reaches, up to the largest that the argument holds: as without a window."""
import pytest
import torch

import gated_delta_rule_34_gb300 as kda

from .test_gpu_cache_ops import BF16, F32, _run_and_check, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, T_q, group, d", [(BF16, 1, 4, 64), (F32, 40, 2, 64), (BF16, 40, 4, 128), (BF16, 300, 1, 64)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 63 - 300, 2 ** 63 - 1])
def test_windows_beyond_any_length(dtype, T_q, group, d, window):
    q, cache, table, lengths = _setup(51, 4, T_q, 2 * group, 2, d, 16, [0, 1, 5, 333], dtype)
    want, want_lse = _run_and_check(q, cache, table, lengths)
    for sinks in (0, 7, 2 ** 31 - 1):
        o, lse = kda.cache_attention(q, cache, table, lengths, window=window, sinks=sinks, return_lse=True)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
