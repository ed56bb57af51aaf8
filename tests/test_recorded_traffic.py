"""The DRAM bytes that the bench line reports for the recurrent kernels: they are reported as long as those kernels' code is
what was profiled.  A change of that code has them captured anew; a change elsewhere must not lose them."""
import pytest

import bench


@pytest.mark.parametrize("kernel", ["chunk_prep", "state_pass", "decode"])
def test_recorded_for_this_code(kernel):
    got = bench.recorded_traffic(kernel)
    assert got is not None, "the kernel's sources are not those of profiles/traffic.json: capture it again (bench.py --ncu)"
    assert got > 0
