"""Thin Python binding of the global-attention operators: rotary positions, the paged
8-bit cache and the attention over it (include/kda.h, "The global-attention layer").

Argument marshalling only, as in ``api``: tensors are checked for device, dtype, shape and
layout, and their data pointers plus the current CUDA stream are handed to ``libkda.so``.
"""
from __future__ import annotations

import contextlib
import math
from typing import NamedTuple

import torch

from .api import _check, _dtype_code, lib

LAYOUTS = {"half": 0, "interleaved": 1}
_NO_SWITCH = contextlib.nullcontext()


def _on(device):
    """Makes ``device`` current for a call, unless it already is."""
    return _NO_SWITCH if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _tensor(name, t, dtype, shape, device):
    """A dense CUDA tensor of this dtype and shape (-1: any size)."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(n >= 0 and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(name, t, like=None):
    """The token stride, in elements, of [..., tokens, H, d] whose [H, d] are dense and whose
    leading dimensions, if any, are token runs one after another."""
    if not t.is_cuda or (like is not None and t.device != like.device):
        raise ValueError(f"{name} must be a CUDA tensor" + ("" if like is None else f" on {like.device}"))
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    h, d = shape[-2], shape[-1]
    if t.numel() == 0:
        return h * d
    if (d > 1 and strides[-1] != 1) or (h > 1 and strides[-2] != d):
        raise ValueError(f"{name}: the heads of a token must be dense")
    stride, span = 0, 0                  # tokens of the inner dimensions, once there are two or more
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if n == 1:
            continue
        if not stride:
            stride, span = s, s * n
        elif s != span:
            raise ValueError(f"{name}: all tokens must be evenly spaced")
        else:
            span *= n
    return stride or h * d


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       trained_len: int = 0, slow_turns: float = 1.0, fast_turns: float = 32.0,
                       device="cuda") -> torch.Tensor:
    """Radians a position of the rot / 2 channel pairs, fp64: base^(-2 i / rot), scaled for
    contexts longer than the trained one:

    "none"      as they are
    "linear"    all divided by ``factor``
    "by_parts"  a pair that makes ``fast_turns`` turns or more over ``trained_len`` positions is
                kept, one that makes ``slow_turns`` or fewer is divided by ``factor``, and
                between them the share of each goes linearly with the turns
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if trained_len <= 0 or not fast_turns > slow_turns:
            raise ValueError("by_parts needs trained_len > 0 and fast_turns > slow_turns")
        turns = trained_len * freq / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / factor)
    elif scaling != "none":
        raise ValueError(f"scaling must be none, linear or by_parts, got {scaling!r}")
    return freq.to(device)


def rotary(q, k, positions, freq, layout: str = "half", amplitude: float = 1.0, q_out=None, k_out=None):
    """Rotary positions through kda_rotary.

    q: [..., H_q, d], k: [..., H_k, d] or None (fp32 or bf16, tokens evenly spaced, heads dense);
    positions: int32, one a token; freq: fp64 [rot / 2] (rotary_frequencies); layout "half" or
    "interleaved".  Returns (q_out, k_out), allocated dense unless given; they may be q and k.
    """
    device, d = q.device, q.shape[-1]
    h_q, n = q.shape[-2], math.prod(q.shape[:-2])
    qs = _rows("q", q)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
    qos = _rows("q_out", q_out, q)
    if q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    ks, kos, h_k, k_ptr, ko_ptr = 0, 0, 0, 0, 0
    if k is not None:
        if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != d:
            raise ValueError(f"k must be [..., H_k, d] of q's tokens, got {tuple(k.shape)} beside {tuple(q.shape)}")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=device)
        if k_out.shape != k.shape:
            raise ValueError("k_out must have k's shape")
        h_k, ks, kos = k.shape[-2], _rows("k", k, q), _rows("k_out", k_out, q)
        k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if positions.numel() != n:
        raise ValueError(f"{n} tokens but {positions.numel()} positions")
    _tensor("positions", positions, torch.int32, positions.shape, device)
    _tensor("freq", freq, torch.float64, (-1,), device)
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be half or interleaved, got {layout!r}")
    with _on(device):
        _check(lib().kda_rotary(q.data_ptr(), qs, q_out.data_ptr(), qos, h_q, k_ptr, ks, ko_ptr, kos, h_k,
                                positions.data_ptr(), freq.data_ptr(), amplitude, n, d, 2 * freq.numel(),
                                LAYOUTS[layout], _dtype_code(q.dtype), _stream(device)))
    return q_out, k_out


class PagedCache(NamedTuple):
    """The pool of a paged 8-bit cache: e4m3 codes [n_pages, H_kv, page, d] and their fp32
    power-of-two scales [n_pages, H_kv], for keys and for values."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def cache_new(n_pages: int, H_kv: int, page: int, d: int, device="cuda") -> PagedCache:
    """An empty pool.  Its contents do not matter until they are written."""
    codes = [torch.zeros((n_pages, H_kv, page, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.ones((n_pages, H_kv), dtype=torch.float32, device=device) for _ in range(2)]
    return PagedCache(*codes, *scales)


def _pool(cache: PagedCache, device):
    """Checks the pool; returns n_pages, H_kv, page, d."""
    shape = cache.k.shape
    _tensor("cache.k", cache.k, torch.float8_e4m3fn, (-1, -1, -1, -1), device)
    _tensor("cache.v", cache.v, torch.float8_e4m3fn, shape, device)
    _tensor("cache.k_scale", cache.k_scale, torch.float32, shape[:2], device)
    _tensor("cache.v_scale", cache.v_scale, torch.float32, shape[:2], device)
    return shape


def cache_write(cache: PagedCache, k, v, block_table, start, cu_seqlens=None) -> PagedCache:
    """New keys and values into the cache, through kda_cache_write; returns the cache.

    k, v: [B, T, H_kv, d], or with cu_seqlens (int32 [N + 1]) packed [1, T_total, H_kv, d] (fp32 or
    bf16, tokens evenly spaced, heads dense); block_table: int32 [N, table_pages];
    start: int32 [N], the position of each sequence's first new token.
    """
    device = k.device
    ks, vs = _rows("k", k), _rows("v", v, k)
    n_pages, h, page, d = _pool(cache, device)
    if k.dim() != 4 or v.shape != k.shape or k.shape[2:] != (h, d):
        raise ValueError(f"k and v must be [B, T, {h}, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    n = _sequences(k.shape[0], cu_seqlens, block_table, start, device)
    with _on(device):
        _check(lib().kda_cache_write(
            k.data_ptr(), ks, v.data_ptr(), vs, cache.k.data_ptr(), cache.v.data_ptr(),
            cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), block_table.data_ptr(), block_table.shape[1],
            start.data_ptr(), 0 if cu_seqlens is None else cu_seqlens.data_ptr(), n, k.shape[1], h, d, n_pages,
            page, _dtype_code(k.dtype), _stream(device)))
    return cache


def _sequences(batch, cu_seqlens, block_table, start, device) -> int:
    n = batch
    if cu_seqlens is not None:
        if batch != 1:
            raise ValueError(f"cu_seqlens requires B == 1 (got {batch})")
        _tensor("cu_seqlens", cu_seqlens, torch.int32, (-1,), device)
        n = cu_seqlens.numel() - 1
        if n < 0:
            raise ValueError("cu_seqlens must not be empty")
    _tensor("block_table", block_table, torch.int32, (n, -1), device)
    _tensor("start", start, torch.int32, (n,), device)
    return n


def cache_read(cache: PagedCache, block_table, start, T: int, cu_seqlens=None, dtype=torch.bfloat16,
               k_out=None, v_out=None):
    """Cached tokens as dense rows, through kda_cache_read: T tokens of each sequence from
    position start[n] on ([N, T, H_kv, d]), or with cu_seqlens those of its packed rows, T rows in
    all ([1, T, H_kv, d]).  Returns (k, v), allocated unless given."""
    device = cache.k.device
    n_pages, h, page, d = _pool(cache, device)
    n = _sequences(block_table.shape[0] if cu_seqlens is None else 1, cu_seqlens, block_table, start, device)
    shape = (n if cu_seqlens is None else 1, T, h, d)
    k = torch.empty(shape, dtype=dtype, device=device) if k_out is None else k_out
    v = torch.empty(shape, dtype=dtype, device=device) if v_out is None else v_out
    _tensor("k_out", k, dtype, shape, device)
    _tensor("v_out", v, dtype, shape, device)
    with _on(device):
        _check(lib().kda_cache_read(
            cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(),
            block_table.data_ptr(), block_table.shape[1], start.data_ptr(),
            0 if cu_seqlens is None else cu_seqlens.data_ptr(), n, T, h, d, n_pages, page, k.data_ptr(), v.data_ptr(),
            _dtype_code(dtype), _stream(device)))
    return k, v


def cache_attention_workspace_size(B: int, T_q: int, H_q: int, H_kv: int, d: int, page: int,
                                   table_pages: int) -> int:
    return int(lib().kda_cache_attention_workspace_size(B, T_q, H_q, H_kv, d, page, table_pages))


def cache_attention(q, cache: PagedCache, block_table, lengths, scale: float | None = None, window: int = 0,
                    sinks: int = 0, out=None, lse=None, return_lse: bool = False, workspace=None):
    """Attention of each sequence's newest tokens over the cache, through kda_cache_attention.

    q: [B, T_q, H_q, d] (fp32 or bf16, tokens evenly spaced, heads dense), the newest T_q tokens, whose
    keys and values are already in the cache; block_table: int32 [B, table_pages]; lengths: int32 [B],
    tokens of each sequence, the newest included; scale: of the scores, 1 / sqrt(d) if None;
    window: a query sees that many tokens back, itself included (0: all), and the first
    ``sinks`` tokens besides.  Returns o [B, T_q, H_q, d], or with return_lse (o, lse) where
    lse is fp32 [B, T_q, H_q].  A workspace of the required size is allocated with torch if none is given.
    """
    device = q.device
    qs = _rows("q", q)
    n_pages, h, page, d = _pool(cache, device)
    if q.dim() != 4 or q.shape[3] != d:
        raise ValueError(f"q must be [B, T_q, H_q, {d}], got {tuple(q.shape)}")
    B, t_q, h_q, _ = q.shape
    _tensor("block_table", block_table, torch.int32, (B, -1), device)
    _tensor("lengths", lengths, torch.int32, (B,), device)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=device)
    else:
        _tensor("out", out, q.dtype, q.shape, device)
    if lse is not None:
        _tensor("lse", lse, torch.float32, (B, t_q, h_q), device)
    elif return_lse:
        lse = torch.empty((B, t_q, h_q), dtype=torch.float32, device=device)
    wide = block_table.shape[1]
    with _on(device):
        if workspace is None:
            need = cache_attention_workspace_size(B, t_q, h_q, h, d, page, wide)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
        elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")
        ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
        _check(lib().kda_cache_attention(
            q.data_ptr(), qs, cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
            cache.v_scale.data_ptr(), block_table.data_ptr(), wide, lengths.data_ptr(), out.data_ptr(),
            0 if lse is None else lse.data_ptr(), B, t_q, h_q, h, d, n_pages, page,
            1.0 / math.sqrt(d) if scale is None else scale, window, sinks, _dtype_code(q.dtype), ws, ws_bytes,
            _stream(device)))
    return (out, lse) if return_lse else out
