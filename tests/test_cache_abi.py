"""The global-attention operators without a GPU: refusals, and the arithmetic that deals out pages.

Every library call here is refused (or has nothing to do) before anything is launched.
"""
import ctypes
import random

import pytest
import torch

import gated_delta_rule_34_gb300 as kda

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_34_gb300 import build
    build.build()
    return kda.lib()


P = 0x10000          # an address that is aligned and never read


def _rotary(L, **kw):
    a = dict(q=P, qs=1024, qo=P, qos=1024, hq=8, k=P, ks=256, ko=P, kos=256, hk=2, pos=P, freq=P, amp=1.0, n=4,
             d=128, rot=128, layout=0, dtype=1)
    a.update(kw)
    return L.kda_rotary(*a.values(), None)


@pytest.mark.parametrize("kw, status", [
    (dict(q=None), INVALID), (dict(q=P + 8), INVALID), (dict(k=None), INVALID), (dict(ko=P + 2), INVALID),
    (dict(pos=None), INVALID), (dict(freq=P + 4), INVALID), (dict(dtype=2), INVALID), (dict(layout=2), INVALID),
    (dict(n=-1), INVALID), (dict(hq=0), INVALID), (dict(hk=-1), INVALID), (dict(d=0), INVALID),
    (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=130), INVALID),
    (dict(qs=1016), INVALID), (dict(qs=1028), INVALID), (dict(kos=128), INVALID),
    (dict(d=260, rot=128, qs=4096, qos=4096, ks=4096, kos=4096), UNSUPPORTED),
    (dict(d=12, rot=12), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED), (dict(n=0), OK), (dict(n=0, q=None), OK),
])
def test_rotary_refusals(L, kw, status):
    assert _rotary(L, **kw) == status
    assert (L.kda_last_error() != b"") == (status != OK)


def _write(L, **kw):
    a = dict(k=P, ks=1024, v=P, vs=1024, kc=P, vc=P, ksc=P, vsc=P, table=P, wide=4, start=P, cu=None, n=2, T=8, h=8,
             d=128, pages=100, page=64, dtype=1)
    a.update(kw)
    return L.kda_cache_write(*a.values(), None)


POOL_REFUSALS = [
    (dict(d=24), UNSUPPORTED), (dict(d=144), UNSUPPORTED), (dict(d=0), INVALID), (dict(h=0), INVALID),
    (dict(page=48), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(pages=-1), INVALID), (dict(pages=1 << 31), UNSUPPORTED), (dict(wide=-1), INVALID), (dict(dtype=9), INVALID),
]


@pytest.mark.parametrize("kw, status", POOL_REFUSALS + [
    (dict(k=None), INVALID), (dict(v=P + 4), INVALID), (dict(kc=None), INVALID), (dict(vc=P + 8), INVALID),
    (dict(ksc=None), INVALID), (dict(vsc=P + 2), INVALID), (dict(table=None), INVALID), (dict(start=None), INVALID),
    (dict(cu=P + 1), INVALID), (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(ks=1000), INVALID),
    (dict(vs=1028), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(n=1 << 28), UNSUPPORTED),
    (dict(T=0), OK), (dict(n=0), OK), (dict(pages=0), OK), (dict(wide=0), OK), (dict(T=0, k=None), OK),
])
def test_write_refusals(L, kw, status):
    assert _write(L, **kw) == status


@pytest.mark.parametrize("kw, status", POOL_REFUSALS + [
    (dict(k=None), INVALID), (dict(v=P + 4), INVALID), (dict(kc=None), INVALID), (dict(start=None), INVALID),
    (dict(table=None), INVALID), (dict(T=0), OK), (dict(n=0), OK),
])
def test_read_refusals(L, kw, status):
    a = dict(kc=P, vc=P, ksc=P, vsc=P, table=P, wide=4, start=P, cu=None, n=2, T=8, h=8, d=128, pages=100, page=64, k=P,
             v=P, dtype=1)
    a.update(kw)
    assert L.kda_cache_read(*a.values(), None) == status


@pytest.mark.parametrize("kw, status", POOL_REFUSALS + [
    (dict(q=None), INVALID), (dict(q=P + 8), INVALID), (dict(o=None), INVALID), (dict(lengths=None), INVALID),
    (dict(table=None), INVALID), (dict(kc=None), INVALID), (dict(lse=P + 2), INVALID), (dict(qs=4000), INVALID),
    (dict(hq=30), INVALID), (dict(hq=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(b=-1), INVALID),
    (dict(b=70000), UNSUPPORTED), (dict(b=60000, tq=60000), UNSUPPORTED), (dict(wide=1 << 27), UNSUPPORTED),
    (dict(b=0), OK), (dict(tq=0), OK), (dict(b=0, q=None), OK),
])
def test_attention_refusals(L, kw, status):
    a = dict(q=P, qs=4096, kc=P, vc=P, ksc=P, vsc=P, table=P, wide=4, lengths=P, o=P, lse=None, b=2, tq=1, hq=32, h=8,
             d=128, pages=100, page=64, scale=0.1, window=0, sinks=0, dtype=1, ws=None, ws_bytes=0)
    a.update(kw)
    assert L.kda_cache_attention(*a.values(), None) == status


def test_attention_refuses_a_short_workspace(L):
    need = L.kda_cache_attention_workspace_size(2, 1, 32, 8, 128, 64, 1024)
    if need == 0:
        pytest.skip("these sizes need no workspace")
    args = [P, 4096, P, P, P, P, P, 1024, P, P, None, 2, 1, 32, 8, 128, 100, 64, 0.1, 0, 0, 1]
    assert L.kda_cache_attention(*args, None, 0, None) == WORKSPACE
    assert L.kda_cache_attention(*args, P, need - 1, None) == WORKSPACE
    assert L.kda_cache_attention(*args, P + 16, need, None) == INVALID


def test_workspace_size_of_what_is_not_taken(L):
    assert L.kda_cache_attention_workspace_size(2, 1, 32, 5, 128, 64, 1024) == 0
    assert L.kda_cache_attention_workspace_size(2, 1, 32, 8, 100, 64, 1024) == 0


# ---------------------------------------------------------------- the binding's own checks

def test_binding_refuses_host_tensors():
    cache = kda.cache_new(4, 2, 16, 32, device="cpu")
    x, i = torch.zeros(1, 3, 2, 32), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: kda.cache_write(cache, x, x, table, i),
                 lambda: kda.cache_read(cache, table, i, 3),
                 lambda: kda.cache_attention(x, cache, table, i),
                 lambda: kda.rotary(x, None, torch.zeros(3, dtype=torch.int32), torch.ones(16, dtype=torch.float64))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rotary_frequencies():
    f = kda.rotary_frequencies(8, base=10000.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(kda.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu"), f / 4.0)
    # turns over 1000 positions: 159, 15.9, 1.59, 0.159; between 1 and 32: kept, part, part, divided
    g = kda.rotary_frequencies(8, scaling="by_parts", factor=4.0, trained_len=1000, device="cpu")
    keep = [1.0, (1000 * 0.1 / 6.283185307179586 - 1) / 31, (1000 * 0.01 / 6.283185307179586 - 1) / 31, 0.0]
    want = [x * (w + (1 - w) / 4) for x, w in zip([1.0, 0.1, 0.01, 0.001], keep)]
    assert torch.allclose(g, torch.tensor(want, dtype=torch.float64), rtol=1e-12)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, scaling="other"), dict(rot=8, scaling="by_parts")):
        with pytest.raises(ValueError):
            kda.rotary_frequencies(device="cpu", **bad)


# ---------------------------------------------------------------- how pages are dealt out

def _first_slot(row, n, page):
    return (row + n * (2 * page - 2)) // page


def _page_run(slot, rows, cu, start, page):
    """The kernels' page_run for a packed batch: (sequence, first row, position, tokens), or None."""
    n_seqs = len(cu) - 1
    lo, hi = 0, n_seqs
    while hi - lo > 1:
        step = (hi - lo + 31) // 32
        last = 0
        for lane in range(32):
            probe = lo + lane * step
            if probe < hi and _first_slot(min(max(cu[probe], 0), rows), probe, page) <= slot:
                last = lane
        lo += last * step
        hi = min(lo + step, hi)
    bos = min(max(cu[lo], 0), rows)
    eos = min(max(cu[lo + 1], bos), rows)
    ordinal = slot - _first_slot(bos, lo, page)
    s = max(start[lo], 0)
    p = s // page + ordinal
    a, b = max(s, p * page), min(s + eos - bos, (p + 1) * page)
    if ordinal < 0 or a >= b:
        return None
    return lo, bos + a - s, a, b - a


@pytest.mark.parametrize("page", [16, 64, 256])
def test_slots_cover_every_new_token_once(page):
    rng = random.Random(page)
    for trial in range(60):
        n = rng.choice([1, 2, 31, 32, 33, 100])
        lens = [rng.choice([0, 1, 2, page - 1, page, page + 1, rng.randint(0, 4 * page)]) for _ in range(n)]
        start = [rng.choice([0, 1, page - 1, page, rng.randint(0, 5 * page)]) for _ in range(n)]
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        rows = cu[-1]
        slots = (rows + n * (2 * page - 2)) // page
        seen = [0] * rows
        pages = set()
        for slot in range(slots):
            run = _page_run(slot, rows, cu, start, page)
            if run is None:
                continue
            seq, row, at, m = run
            assert (seq, at // page) not in pages and at // page == (at + m - 1) // page
            pages.add((seq, at // page))
            for j in range(m):
                assert cu[seq] <= row + j < cu[seq + 1] and at + j - start[seq] == row + j - cu[seq]
                seen[row + j] += 1
        assert seen == [1] * rows


@pytest.mark.parametrize("page", [16, 64])
def test_malformed_offsets_stay_in_bounds(page):
    rng = random.Random(7 * page)
    for trial in range(200):
        n, rows = rng.randint(1, 70), rng.randint(1, 500)
        cu = [rng.choice([rng.randint(-50, 600), -2 ** 31, 2 ** 31 - 1]) for _ in range(n + 1)]
        start = [rng.choice([rng.randint(-50, 600), -2 ** 31, 2 ** 31 - 1]) for _ in range(n)]
        for slot in range((rows + n * (2 * page - 2)) // page):
            run = _page_run(slot, rows, cu, start, page)
            if run is not None:
                assert 0 <= run[1] and run[1] + run[3] <= rows and run[2] >= 0 and 1 <= run[3] <= page


@pytest.mark.parametrize("page", [16, 128])
def test_fixed_length_slots_suffice(page):
    for T in list(range(1, 3 * page)):
        slots = (T + 2 * page - 2) // page
        for start in (0, 1, page // 2, page - 1):
            assert (start + T - 1) // page - start // page + 1 <= slots
