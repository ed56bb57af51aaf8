"""Thin Python binding of the global-attention operators: rotary positions, the paged
8-bit cache, its pages' sharing and the attention over it (include/kda.h, "The global-attention layer").

Argument marshalling only, as in ``api``: tensors are checked for device, dtype, shape and
layout, and their data pointers plus the current CUDA stream are handed to ``libkda.so``.
A decode step's kernels take a few microseconds, so the marshalling itself is compiled
(csrc/cache_binding.cpp): a call that it finds well formed is launched, for any other it returns
None and launches nothing, and what is wrong is then looked for here.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os
from importlib.machinery import ExtensionFileLoader
from typing import NamedTuple

import torch

from . import build as _build
from .api import _check, _dtype_code, lib

E4M3, F32, F64, I32 = torch.float8_e4m3fn, torch.float32, torch.float64, torch.int32


@functools.lru_cache(maxsize=None)
def _binding():
    """The compiled marshalling, calling the library that ``lib`` has loaded; raises if it has not been built."""
    entries = [getattr(lib(), name) for name in ("kda_rotary", "kda_cache_write", "kda_cache_read",
                                                 "kda_cache_attention", "kda_cache_attention_workspace_size",
                                                 "kda_cache_copy", "kda_cache_resize", "kda_cache_fork",
                                                 "kda_cache_compact", "kda_cache_pages_workspace_size",
                                                 "kda_cache_attention_shared",
                                                 "kda_cache_attention_shared_workspace_size")]
    if not os.path.exists(_build.BINDING):
        raise RuntimeError(
            f"KDA binding not found at {_build.BINDING}; build it with "
            "`python -m gated_delta_rule_34_gb300.build` (there is no fallback path)")
    loader = ExtensionFileLoader("kda_cache_binding", _build.BINDING)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
    loader.exec_module(module)
    module.bind(*(ctypes.cast(e, ctypes.c_void_p).value for e in entries), _check)
    return module


def _is_elsewhere(index: int) -> bool:
    """Whether device ``index`` is another than the current one."""
    if index < 0:
        raise ValueError("the global-attention operators take CUDA tensors")
    return index != torch.cuda.current_device()


def _not_understood(name: str):
    raise TypeError(f"{name}: arguments of a type or size that it does not take")


def _tensor(name, t, dtype, shape, index):
    """A dense CUDA tensor of this dtype and shape (-1: any size) on device ``index``."""
    if t.dtype is dtype and t.get_device() == index >= 0 and t.is_contiguous() and t.shape == shape:
        return
    if index < 0 or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{index}" if index >= 0 else ""))
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(n >= 0 and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(name, t, dtype, index):
    """[..., tokens, H, d] whose [H, d] are dense and whose tokens are evenly spaced, leading
    dimensions being token runs one after another."""
    if index < 0 or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{index}" if index >= 0 else ""))
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) < 3:
        raise ValueError(f"{name} must be [..., tokens, H, d], got {tuple(shape)}")
    h, d = shape[-2:]
    if t.is_contiguous():
        return
    strides = t.stride()
    if (d > 1 and strides[-1] != 1) or (h > 1 and strides[-2] != d):
        raise ValueError(f"{name}: the heads of a token must be dense")
    stride, span = None, 0               # of the inner dimensions' tokens, once there are two or more
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if n == 1:
            continue
        if stride is None:
            stride, span = s, s * n
        elif s != span:
            raise ValueError(f"{name}: all tokens must be evenly spaced")
        else:
            span *= n
    if stride is not None and stride < h * d:
        raise ValueError(f"{name}: tokens must not overlap")


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
    done = _binding().rotary(q, k, positions, freq, layout, amplitude, q_out, k_out)
    if done is not None:
        return done
    index = q.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return rotary(q, k, positions, freq, layout, amplitude, q_out, k_out)
    shape, dtype = q.shape, q.dtype
    _dtype_code(dtype)
    _rows("q", q, dtype, index)
    h_q, d = shape[-2:]
    n = q.numel() // (h_q * d) if h_q * d else 0
    if q_out is not None:
        _rows("q_out", q_out, dtype, index)
        if q_out.shape != shape:
            raise ValueError("q_out must have q's shape")
    if k is not None:
        _rows("k", k, dtype, index)
        if k.shape[:-2] != shape[:-2] or k.shape[-1] != d:
            raise ValueError(f"k must be [..., H_k, d] of q's tokens, got {tuple(k.shape)} beside {tuple(shape)}")
        if k_out is not None:
            _rows("k_out", k_out, dtype, index)
            if k_out.shape != k.shape:
                raise ValueError("k_out must have k's shape")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if positions.numel() != n:
        raise ValueError(f"{n} tokens but {positions.numel()} positions")
    _tensor("positions", positions, I32, positions.shape, index)
    _tensor("freq", freq, F64, (-1,) if freq.dim() != 1 else freq.shape, index)
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout must be half or interleaved, got {layout!r}")
    _not_understood("rotary")


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


def _pool(cache: PagedCache, index):
    """Checks the pool; returns n_pages, H_kv, page, d."""
    k, v, k_scale, v_scale = cache
    shape = k.shape
    blocks = shape[:2]
    if not (k.dtype is E4M3 and v.dtype is E4M3 and k_scale.dtype is F32 and v_scale.dtype is F32
            and k.get_device() == v.get_device() == k_scale.get_device() == v_scale.get_device() == index >= 0
            and len(shape) == 4 and v.shape == shape and k_scale.shape == blocks and v_scale.shape == blocks
            and k.is_contiguous() and v.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()):
        _tensor("cache.k", k, E4M3, (-1, -1, -1, -1), index)
        _tensor("cache.v", v, E4M3, shape, index)
        _tensor("cache.k_scale", k_scale, F32, blocks, index)
        _tensor("cache.v_scale", v_scale, F32, blocks, index)
    return shape


def _sequences(batch, cu_seqlens, block_table, start, index) -> int:
    n = batch
    if cu_seqlens is not None:
        if batch != 1:
            raise ValueError(f"cu_seqlens requires B == 1 (got {batch})")
        n = cu_seqlens.numel() - 1
        if n < 0:
            raise ValueError("cu_seqlens must not be empty")
        _tensor("cu_seqlens", cu_seqlens, I32, (n + 1,), index)
    _tensor("block_table", block_table, I32, (n, block_table.shape[-1]), index)
    _tensor("start", start, I32, (n,), index)
    return n


def cache_write(cache: PagedCache, k, v, block_table, start, cu_seqlens=None) -> PagedCache:
    """New keys and values into the cache, through kda_cache_write; returns the cache.

    k, v: [B, T, H_kv, d], or with cu_seqlens (int32 [N + 1]) packed [1, T_total, H_kv, d] (fp32 or
    bf16, tokens evenly spaced, heads dense); block_table: int32 [N, table_pages];
    start: int32 [N], the position of each sequence's first new token.  No page that is written to may have another
    holder: a row cut inside a page that it shares parts from it first, see cache_fork.
    """
    done = _binding().cache_write(cache, k, v, block_table, start, cu_seqlens)
    if done is not None:
        return done
    index = k.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_write(cache, k, v, block_table, start, cu_seqlens)
    shape, dtype = k.shape, k.dtype
    _dtype_code(dtype)
    _rows("k", k, dtype, index)
    _rows("v", v, dtype, index)
    n_pages, h, page, d = _pool(cache, index)
    if len(shape) != 4 or v.shape != shape or shape[2] != h or shape[3] != d:
        raise ValueError(f"k and v must be [B, T, {h}, {d}], got {tuple(shape)} and {tuple(v.shape)}")
    _sequences(shape[0], cu_seqlens, block_table, start, index)
    _not_understood("cache_write")


def cache_read(cache: PagedCache, block_table, start, T: int, cu_seqlens=None, dtype=torch.bfloat16,
               k_out=None, v_out=None):
    """Cached tokens as dense rows, through kda_cache_read: T tokens of each sequence from
    position start[n] on ([N, T, H_kv, d]), or with cu_seqlens those of its packed rows, T rows in
    all ([1, T, H_kv, d]).  Returns (k, v), allocated unless given."""
    done = _binding().cache_read(cache, block_table, start, T, cu_seqlens, dtype, k_out, v_out)
    if done is not None:
        return done
    index = cache[0].get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_read(cache, block_table, start, T, cu_seqlens, dtype, k_out, v_out)
    _dtype_code(dtype)
    n_pages, h, page, d = _pool(cache, index)
    n = _sequences(block_table.shape[0] if cu_seqlens is None else 1, cu_seqlens, block_table, start, index)
    shape = (n if cu_seqlens is None else 1, T, h, d)
    if k_out is not None:
        _tensor("k_out", k_out, dtype, shape, index)
    if v_out is not None:
        _tensor("v_out", v_out, dtype, shape, index)
    _not_understood("cache_read")


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
    done = _binding().cache_attention(q, cache, block_table, lengths, scale, window, sinks, out, lse, return_lse, workspace)
    if done is not None:
        return done
    index = q.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_attention(q, cache, block_table, lengths, scale, window, sinks, out, lse, return_lse, workspace)
    shape, dtype = q.shape, q.dtype
    _dtype_code(dtype)
    _rows("q", q, dtype, index)
    n_pages, h, page, d = _pool(cache, index)
    if len(shape) != 4 or shape[3] != d:
        raise ValueError(f"q must be [B, T_q, H_q, {d}], got {tuple(shape)}")
    _tensor("block_table", block_table, I32, (shape[0], block_table.shape[-1]), index)
    _tensor("lengths", lengths, I32, (shape[0],), index)
    if out is not None:
        _tensor("out", out, dtype, shape, index)
    if lse is not None:
        _tensor("lse", lse, F32, shape[:3], index)
    if workspace is not None and (workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {q.device}")
    _not_understood("cache_attention")


def cache_attention_shared_workspace_size(B: int, T_q: int, H_q: int, H_kv: int, d: int, page: int, table_pages: int,
                                          prefix_pages: int, n_groups: int) -> int:
    return int(lib().kda_cache_attention_shared_workspace_size(B, T_q, H_q, H_kv, d, page, table_pages, prefix_pages, n_groups))


def cache_attention_shared(q, cache: PagedCache, block_table, lengths, prefix_table, prefix_lengths, cu_groups,
                           scale: float | None = None, out=None, lse=None, return_lse: bool = False, workspace=None):
    """cache_attention (without a window) for sequences in groups that share a prefix, which is read once for each group,
    through kda_cache_attention_shared.

    q, cache, block_table, lengths, scale, out, lse, return_lse, workspace: as in cache_attention; the rows of block_table hold
    each sequence from its first token on, as cache_fork leaves them.  prefix_table: int32 [G, prefix_pages], the pages of each
    group's prefix; prefix_lengths: int32 [G], its tokens, of which whole pages are shared; cu_groups: int32 [G + 1], group g
    is sequences cu_groups[g] .. cu_groups[g + 1] - 1.  A sequence some of whose queries do not see all of the prefix attends
    over its own row alone, and so do all where the sizes leave too little to share; these go by the prefix table's width, which had
    better be no more than the longest prefix needs.
    """
    done = _binding().cache_attention_shared(q, cache, block_table, lengths, prefix_table, prefix_lengths, cu_groups, scale, out, lse,
                                             return_lse, workspace)
    if done is not None:
        return done
    index = q.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_attention_shared(q, cache, block_table, lengths, prefix_table, prefix_lengths, cu_groups, scale, out, lse,
                                          return_lse, workspace)
    shape, dtype = q.shape, q.dtype
    _dtype_code(dtype)
    _rows("q", q, dtype, index)
    n_pages, h, page, d = _pool(cache, index)
    if len(shape) != 4 or shape[3] != d:
        raise ValueError(f"q must be [B, T_q, H_q, {d}], got {tuple(shape)}")
    _tensor("block_table", block_table, I32, (shape[0], block_table.shape[-1]), index)
    _tensor("lengths", lengths, I32, (shape[0],), index)
    _tensor("prefix_table", prefix_table, I32, (-1, -1), index)
    _tensor("prefix_lengths", prefix_lengths, I32, prefix_table.shape[:1], index)
    _tensor("cu_groups", cu_groups, I32, (prefix_table.shape[0] + 1,), index)
    if out is not None:
        _tensor("out", out, dtype, shape, index)
    if lse is not None:
        _tensor("lse", lse, F32, shape[:3], index)
    _workspace(workspace, index)
    _not_understood("cache_attention_shared")


def _workspace(workspace, index):
    if workspace is not None and (workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{index}")


def cache_copy(cache: PagedCache, src, dst) -> PagedCache:
    """Page src[i] copied to page dst[i], codes and scales of all heads, through kda_cache_copy; returns the cache.

    src, dst: int32 [n]; pairs with an entry outside [0, n_pages) (-1) are skipped.  No page may be the target of two pairs, or of
    one and the source of another.
    """
    done = _binding().cache_copy(cache, src, dst)
    if done is not None:
        return done
    index = src.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_copy(cache, src, dst)
    _pool(cache, index)
    _tensor("src", src, I32, (-1,), index)
    _tensor("dst", dst, I32, src.shape, index)
    _not_understood("cache_copy")


def cache_pages_workspace_size(n_pages: int, n_rows: int) -> int:
    return int(lib().kda_cache_pages_workspace_size(n_pages, n_rows))


def cache_resize(refs, block_table, rows, tokens, page: int, missing=None, workspace=None):
    """The listed rows of the block table brought to the pages that their tokens need, through kda_cache_resize: pages past
    these are given back, missing ones taken, the lowest free ones first.  In place.

    refs: int32 [n_pages], how many entries hold each page (a new pool: torch.zeros); block_table: int32 [n_rows, table_pages];
    rows, tokens: int32 [n]; page: tokens of a page.  Returns missing, int32 [1]: pages wanted when the pool had no more
    (their entries are -1).  A workspace of the required size is allocated with torch if none is given.
    """
    done = _binding().cache_resize(refs, block_table, rows, tokens, page, missing, workspace)
    if done is not None:
        return done
    index = rows.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_resize(refs, block_table, rows, tokens, page, missing, workspace)
    _tensor("refs", refs, I32, (-1,), index)
    _tensor("block_table", block_table, I32, (-1, -1), index)
    _tensor("rows", rows, I32, (-1,), index)
    _tensor("tokens", tokens, I32, rows.shape, index)
    if missing is not None:
        _tensor("missing", missing, I32, (1,), index)
    _workspace(workspace, index)
    _not_understood("cache_resize")


def cache_fork(refs, block_table, lengths, src, dst, page: int, from_pages=None, to_pages=None, missing=None, workspace=None):
    """Rows dst[i] of the block table become the sequences of rows src[i], through kda_cache_fork: full pages are shared, a
    partly filled last page is replaced by a free one.  In place; dst rows must hold nothing (cache_resize to 0 gives back).

    refs, block_table, page: as in cache_resize; lengths: int32 [n_rows], tokens of each row (dst's are set; with less for a source
    than it has, the branch begins earlier); src, dst: int32 [n], a source may stand in many pairs.  Returns (from_pages, to_pages, missing): the pages to copy, int32 [n], -1 where there is none
    (cache_copy, for the pool of each layer that has this table), and int32 [1], pages wanted when the pool had no more.

    A row taken back to a length inside a page that it shares must not be written to, for its other holders' sake.  It goes on as its
    own fork: its lengths entry set, cache_fork to a row that holds nothing, cache_copy, then cache_resize of the old row to 0.  The
    states of recurrent layers are the caller's to copy.
    """
    done = _binding().cache_fork(refs, block_table, lengths, src, dst, page, from_pages, to_pages, missing, workspace)
    if done is not None:
        return done
    index = src.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_fork(refs, block_table, lengths, src, dst, page, from_pages, to_pages, missing, workspace)
    _tensor("refs", refs, I32, (-1,), index)
    _tensor("block_table", block_table, I32, (-1, -1), index)
    _tensor("lengths", lengths, I32, block_table.shape[:1], index)
    _tensor("src", src, I32, (-1,), index)
    _tensor("dst", dst, I32, src.shape, index)
    for name, t, n in (("from_pages", from_pages, src.numel()), ("to_pages", to_pages, src.numel()), ("missing", missing, 1)):
        if t is not None:
            _tensor(name, t, I32, (n,), index)
    _workspace(workspace, index)
    _not_understood("cache_fork")


def cache_compact(refs, block_table, refs_out=None, table_out=None, page_map=None, from_pages=None, to_pages=None, held=None):
    """The held pages brought to the front of the pool, through kda_cache_compact: refs and the block table are changed in
    place, or written to refs_out and table_out where these are given.

    Returns (page_map, from_pages, to_pages, held): int32 [n_pages], where each held page is now (-1: not held), for other tables;
    int32 [n_pages // 2], the pages to copy (cache_copy, for the pool of each layer that has this table), -1 past the last; int32 [1],
    how many pages are held.
    """
    done = _binding().cache_compact(refs, block_table, refs_out, table_out, page_map, from_pages, to_pages, held)
    if done is not None:
        return done
    index = refs.get_device()
    if _is_elsewhere(index):
        with torch.cuda.device(index):
            return cache_compact(refs, block_table, refs_out, table_out, page_map, from_pages, to_pages, held)
    _tensor("refs", refs, I32, (-1,), index)
    _tensor("block_table", block_table, I32, (-1, -1), index)
    n = refs.numel()
    for name, t, shape in (("refs_out", refs_out, refs.shape), ("table_out", table_out, block_table.shape), ("page_map", page_map, (n,)),
                           ("from_pages", from_pages, (n // 2,)), ("to_pages", to_pages, (n // 2,)), ("held", held, (1,))):
        if t is not None:
            _tensor(name, t, I32, shape, index)
    _not_understood("cache_compact")
