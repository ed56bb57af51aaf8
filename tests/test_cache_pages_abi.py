"""Pages shared, taken, given back and moved, without a GPU: refusals of the C entries, and calls with nothing to do."""
import inspect

import pytest
import torch

import gated_delta_rule_34_gb300 as kda
from gated_delta_rule_34_gb300 import cache

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = 0x10000          # an address that is aligned and never read


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_34_gb300 import build
    build.build()
    return kda.lib()


@pytest.mark.parametrize("kw, status", [
    (dict(kc=None), INVALID), (dict(vc=P + 8), INVALID), (dict(ksc=P + 2), INVALID), (dict(vsc=None), INVALID),
    (dict(src=None), INVALID), (dict(dst=P + 1), INVALID), (dict(n=-1), INVALID), (dict(h=0), INVALID),
    (dict(d=24), UNSUPPORTED), (dict(d=144), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(pages=-1), INVALID),
    (dict(pages=1 << 31), UNSUPPORTED), (dict(n=1 << 29, h=8), UNSUPPORTED), (dict(n=0), OK), (dict(n=0, src=None), OK),
    (dict(pages=0, kc=None), OK),
])
def test_copy_refusals(L, kw, status):
    a = dict(kc=P, vc=P, ksc=P, vsc=P, src=P, dst=P, n=4, h=8, d=128, pages=100, page=64)
    a.update(kw)
    assert L.kda_cache_copy(*a.values(), None) == status


ROWS = [(dict(refs=None), INVALID), (dict(table=P + 2), INVALID), (dict(pages=-1), INVALID), (dict(n_rows=-1), INVALID),
        (dict(wide=-1), INVALID), (dict(n=-1), INVALID), (dict(n=65537), UNSUPPORTED), (dict(page=100), UNSUPPORTED),
        (dict(pages=1 << 31), UNSUPPORTED), (dict(wide=1 << 26), UNSUPPORTED), (dict(n=65536, wide=32768), UNSUPPORTED),
        (dict(missing=P + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=256), WORKSPACE), (dict(ws=P + 128), INVALID)]


@pytest.mark.parametrize("kw, status", ROWS + [
    (dict(rows=None), INVALID), (dict(tokens=P + 1), INVALID), (dict(n=0, missing=None, rows=None), OK),
    (dict(wide=0, missing=None, table=None), OK), (dict(n_rows=0, missing=None, table=None), OK),
])
def test_resize_refusals(L, kw, status):
    a = dict(refs=P, pages=100, table=P, n_rows=4, wide=8, rows=P, tokens=P, n=3, page=64, missing=P, ws=P, ws_bytes=1 << 19)
    a.update(kw)
    assert L.kda_cache_resize(*a.values(), None) == status


@pytest.mark.parametrize("kw, status", ROWS + [
    (dict(lengths=None), INVALID), (dict(src=None), INVALID), (dict(dst=P + 2), INVALID), (dict(to=None), INVALID),
    (dict(frm=P + 2), INVALID), (dict(n=0, missing=None, src=None), OK),
])
def test_fork_refusals(L, kw, status):
    a = dict(refs=P, pages=100, table=P, n_rows=4, wide=8, lengths=P, src=P, dst=P, n=3, page=64, frm=P, to=P, missing=P,
             ws=P, ws_bytes=1 << 19)
    a.update(kw)
    assert L.kda_cache_fork(*a.values(), None) == status


@pytest.mark.parametrize("kw, status", [
    (dict(refs=None), INVALID), (dict(refs_out=P + 1), INVALID), (dict(table=None), INVALID), (dict(table_out=P + 2), INVALID),
    (dict(map=None), INVALID), (dict(frm=None), INVALID), (dict(to=P + 2), INVALID), (dict(held=None), INVALID),
    (dict(pages=-1), INVALID), (dict(n_rows=-1), INVALID), (dict(wide=-1), INVALID), (dict(pages=(1 << 31) - 1), UNSUPPORTED),
    (dict(n_rows=1 << 30, wide=1 << 8), UNSUPPORTED),
])
def test_compact_refusals(L, kw, status):
    a = dict(refs=P, refs_out=P, pages=100, table=P, table_out=P, n_rows=4, wide=8, map=P, frm=P, to=P, held=P)
    a.update(kw)
    assert L.kda_cache_compact(*a.values(), None) == status


@pytest.mark.parametrize("kw, status", [
    (dict(q=None), INVALID), (dict(o=P + 4), INVALID), (dict(lengths=None), INVALID), (dict(table=None), INVALID),
    (dict(prefix=None), INVALID), (dict(prefix_len=P + 2), INVALID), (dict(cu=None), INVALID), (dict(prefix_pages=-1), INVALID),
    (dict(groups=-1), INVALID), (dict(groups=3), INVALID), (dict(prefix_pages=1 << 26), UNSUPPORTED), (dict(dtype=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(hq=9), INVALID), (dict(d=136), UNSUPPORTED), (dict(qs=1028), INVALID),
    (dict(B=65536), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=256), WORKSPACE), (dict(ws=P + 128), INVALID),
    (dict(B=0, groups=0), OK), (dict(T_q=0), OK), (dict(lse=P + 1), INVALID),
])
def test_shared_refusals(L, kw, status):
    a = dict(q=P, qs=1024, kc=P, vc=P, ksc=P, vsc=P, table=P, wide=8, lengths=P, prefix=P, prefix_pages=4000, prefix_len=P, cu=P,
             groups=1, o=P, lse=None, B=2, T_q=1, hq=8, hkv=2, d=128, pages=100, page=64, scale=1.0, dtype=1, ws=P,
             ws_bytes=1 << 40)
    a.update(kw)
    assert L.kda_cache_attention_shared(*a.values(), None) == status


def test_shared_workspace_size(L):
    size = kda.cache_attention_shared_workspace_size
    rows = 4 * 3 * 8
    assert size(4, 3, 8, 2, 128, 64, 10, 2000, 2) >= rows * (16 + 512)
    # nothing to share, or too little
    assert size(4, 3, 8, 2, 128, 64, 10, 0, 2) == size(4, 3, 8, 2, 128, 64, 10, 5, 2) == size(4, 3, 8, 2, 128, 64, 10, 5, 0) == kda.cache_attention_workspace_size(4, 3, 8, 2, 128, 64, 10)
    assert size(4, 3, 8, 3, 128, 64, 10, 5, 2) == size(4, 3, 8, 2, 128, 64, 10, 5, 5) == size(0, 3, 8, 2, 128, 64, 10, 5, 0) == 0


def test_workspace_size(L):
    size = kda.cache_pages_workspace_size
    assert size(0, 0) >= 4 * 65536 and size(0, 0) % 256 == 0   # (places of 65536 units of rows)
    assert size(1000, 24) >= size(0, 0) + 4096 - 256
    assert size((1 << 31) - 1, 5) > 1 << 33
    assert size(-1, 4) == size(1 << 31, 4) == size(4, -1) == 0


@pytest.mark.parametrize("name", ["cache_copy", "cache_resize", "cache_fork", "cache_compact", "cache_attention_shared"])
def test_odd_arguments_are_left_alone(L, name):
    entry, public = getattr(cache._binding(), name), getattr(kda, name)
    n = len(inspect.signature(public).parameters)
    assert entry(*[None] * n) is None
    x = torch.zeros(4, dtype=torch.int32)
    for i in range(n):
        assert entry(*[x if j == i else None for j in range(n)]) is None
    assert entry(*[x] * n) is None
    assert entry(*[(x, x, x, x)] * n) is None
    with pytest.raises(TypeError, match="arguments"):
        entry(*[None] * (n + 1))


def test_public_calls_name_what_is_wrong(L):
    pool = kda.cache_new(2, 4, 16, 64, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: kda.cache_copy(pool, i, i), lambda: kda.cache_resize(i, i[None], i, i, 16),
                 lambda: kda.cache_fork(i, i[None], i, i, i, 16), lambda: kda.cache_compact(i, i[None]),
                 lambda: kda.cache_attention_shared(torch.zeros(1, 1, 4, 64), pool, i[None], i, i[None], i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
