"""The largest number of query rows of the attention over the cache, without a GPU: what is taken has a workspace of a
sensible size, what is not is refused."""
import pytest

import gated_delta_rule_34_gb300 as kda

P = 0x10000
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_34_gb300 import build
    build.build()
    return kda.lib()


@pytest.mark.parametrize("d", [16, 128])
@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 31 - 200])
def test_row_tiles_do_not_overflow(L, rows, d):
    assert L.kda_cache_attention_workspace_size(1, rows, 1, 1, d, 16, 1024) == 0
    args = [P, d, P, P, P, P, P, 1024, P, P, None, 1, rows, 1, 1, d, 100, 16, 0.1, 0, 0, 1]
    assert L.kda_cache_attention(*args, None, 0, None) == UNSUPPORTED


@pytest.mark.parametrize("rows", [2 ** 31 - 256, 2 ** 30, 5000])
def test_workspace_of_many_rows(L, rows):
    assert L.kda_cache_attention_workspace_size(1, rows, 1, 1, 16, 16, 1024) < 2 ** 30
