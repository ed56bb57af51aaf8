"""The self-test of the many-row attention's waits, without a GPU: what it refuses."""
import pytest

import gated_delta_rule_34_gb300 as kda


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_delta_rule_34_gb300 import build
    build.build()


@pytest.mark.parametrize("args", [(-1, 0, 1), (0, -1, 1), (0, 0, -1), (0, 0, 2_000_001)])
def test_refusals(args):
    with pytest.raises(kda.KDAError):
        kda.selftest_attention_stall(*args)


def test_on_and_off():
    kda.selftest_attention_stall(3, 4, 1000)
    kda.selftest_attention_stall()
