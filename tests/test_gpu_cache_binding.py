"""The compiled marshalling of the global-attention operators on the GPU: what it returns, its errors, its workspace."""
import pytest
import torch

import gated_delta_rule_34_gb300 as kda

pytestmark = pytest.mark.gpu


def _case(dtype=torch.bfloat16, B=2, H=4, d=64, page=16):
    torch.manual_seed(5)
    pool = kda.cache_new(2 * B, H, page, d)
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    k = torch.randn(B, 2 * page, H, d, device="cuda").to(dtype)
    kda.cache_write(pool, k, k, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    q = torch.randn(B, 1, 2 * H, d, device="cuda").to(dtype)
    return q, pool, table, torch.full((B,), 2 * page - 3, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_given_tensors_come_back(dtype):
    q, pool, table, lengths = _case(dtype)
    o, lse = kda.cache_attention(q, pool, table, lengths, return_lse=True)
    out, mine = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    got = kda.cache_attention(q, pool, table, lengths, out=out, lse=mine)
    assert got is out and torch.equal(out, o) and torch.equal(mine, lse)
    got = kda.cache_attention(q, pool, table, lengths, out=out, lse=mine, return_lse=True)
    assert got[0] is out and got[1] is mine
    assert kda.cache_write(pool, q[:, :, :4], q[:, :, 4:], table, lengths) is pool
    k, v = kda.cache_read(pool, table, lengths, 1, dtype=dtype)
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    got = kda.cache_read(pool, table, lengths, 1, dtype=dtype, k_out=k_out, v_out=v_out)
    assert got[0] is k_out and got[1] is v_out and torch.equal(k, k_out) and torch.equal(v, v_out)
    freq = kda.rotary_frequencies(64)
    one, two = kda.rotary(q, None, lengths, freq)
    assert two is None and kda.rotary(q, None, lengths, freq, q_out=out)[0] is out and torch.equal(one, out)


def test_errors_of_the_library_are_raised():
    q, pool, table, lengths = _case()
    need = kda.cache_attention_workspace_size(2, 1, 8, 4, 64, 16, 2)
    with pytest.raises(kda.KDAError):
        kda.cache_attention(q, pool, table, lengths, window=-1)
    if need:
        with pytest.raises(kda.KDAError):
            kda.cache_attention(q, pool, table, lengths, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    for odd in (dict(window=2 ** 63), dict(sinks=2 ** 31)):
        with pytest.raises(OverflowError):
            kda.cache_attention(q, pool, table, lengths, **odd)
    for odd in (dict(window="all"), dict(scale="none"), dict(sinks=1.5)):
        with pytest.raises(TypeError):
            kda.cache_attention(q, pool, table, lengths, **odd)
    with pytest.raises(RuntimeError):                      # a result of negative size: torch's own refusal
        kda.cache_read(pool, table, lengths, -1)
    with pytest.raises(TypeError):
        kda.cache_attention(q.half(), pool, table, lengths)
    with pytest.raises(TypeError):
        kda.cache_read(pool, table, lengths, 1, dtype=torch.float16)
    kda.cache_attention(q, pool, table, lengths)           # and nothing is left behind


def test_results_belong_to_the_current_stream():
    """Results and workspace are allocated on the stream that the kernels run on."""
    q, pool, table, lengths = _case()
    want = kda.cache_attention(q, pool, table, lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(50):
            got = kda.cache_attention(q, pool, table, lengths)
            assert not got.requires_grad
    side.synchronize()
    assert torch.equal(got, want)


def test_memory_is_given_back():
    q, pool, table, lengths = _case()
    kda.cache_attention(q, pool, table, lengths, return_lse=True)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(20):
        kda.cache_attention(q, pool, table, lengths, return_lse=True)
        kda.rotary(q, q, lengths, kda.rotary_frequencies(64))
        kda.cache_read(pool, table, lengths, 1)
    assert torch.cuda.memory_allocated() == before
