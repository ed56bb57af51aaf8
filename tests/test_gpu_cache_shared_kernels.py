"""Which kernels a shared-attention call launches, so that the tests of each reach it."""
import pytest
import torch

from .test_gpu_cache_shared import BF16, F32, WIDE, WIDE32, Case

pytestmark = pytest.mark.gpu

PREFIX_TC, TC, ROWS = "prefix_tc_kernel", "attention_tc_kernel", ("attention_whole_kernel", "attention_share_kernel")
PREFIX, REST = "Part)1", "Part)2"                          # of a kernel's template arguments


def kernels(case):
    """The names of a call's kernels."""
    case.run()
    torch.cuda.synchronize()
    for _ in range(5):                                     # (a process's first trace may be empty)
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as trace:
            case.run()
            torch.cuda.synchronize()
        names = [e.name for e in trace.events() if "kda::" in e.name]
        if names:
            return names
    pytest.skip("kernels cannot be traced here")


def launched(names, kernel, part=""):
    return any(k in name and part in name for name in names for k in ((kernel,) if isinstance(kernel, str) else kernel))


@pytest.mark.parametrize("dtype, T_q, hq, hk, d, n, more, prefix, rest", [
    (BF16, 1, 4, 2, 64, 3, 0, None, ROWS),                 # nothing to gain
    (F32, 1, 4, 2, 64, 70, 0, None, ROWS),
    (WIDE, 1, 4, 2, 64, 3, 0, ROWS, ROWS),                 # few rows a group
    (WIDE, 1, 4, 2, 64, 70, 0, PREFIX_TC, ROWS),           # many
    (WIDE, 1, 8, 1, 128, 20, 0, PREFIX_TC, ROWS),
    (WIDE, 33, 8, 2, 128, 3, 0, PREFIX_TC, ROWS),          # many rows a sequence, little room behind the prefix,
    (WIDE, 33, 8, 2, 128, 3, 1, PREFIX_TC, TC),     # and much
    (WIDE32, 1, 4, 2, 64, 3, 0, ROWS, ROWS),
    (WIDE32, 1, 4, 2, 64, 70, 0, ROWS, ROWS),
])
def test_kernels(dtype, T_q, hq, hk, d, n, more, prefix, rest):
    case = Case(30, T_q, hq, hk, d, 32, dtype, [(300, [T_q + i % 40 for i in range(n)])])
    if more:                                               # 1,280 tokens: the block table wider than the prefix's
        wide = case.prefix_table.shape[1] + 40
        case.table = torch.nn.functional.pad(case.table, (0, wide - case.table.shape[1]), value=-1)
    names = kernels(case)
    assert launched(names, PREFIX_TC) == (prefix == PREFIX_TC)
    assert launched(names, ROWS, PREFIX) == (prefix == ROWS)
    if prefix is None:
        assert launched(names, ROWS) and not launched(names, REST)
    else:
        assert launched(names, TC if rest == TC else ROWS, REST) and not launched(names, ROWS if rest == TC else TC, REST)


@pytest.mark.parametrize("longest, tc", [(1000, False), (1024, False), (1025, True)])
def test_nothing_shared_by_many_rows(longest, tc):
    names = kernels(Case(31, 9, 4, 2, 128, 32, BF16, [], before=[longest, 9]))
    assert launched(names, TC) == tc and launched(names, ROWS, REST) != tc and not launched(names, PREFIX_TC)
