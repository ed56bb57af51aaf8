"""GB300 (sm_103a) Kimi Delta Attention layer: a C-ABI CUDA library plus a thin binding.

    from gated_delta_rule_34_gb300 import chunk_prefill, decode_step, gate

The binding loads ``_build/libkda.so`` on first use (build it with
``python -m gated_delta_rule_34_gb300.build``); importing the package loads
nothing, so the seeded input generator (``.inputs``) can be used without a GPU.
"""
from .api import (KDAError, auto_segments, chunk_prefill, chunk_prefill_from_host,  # noqa: F401
                  chunk_prefill_segmented, chunk_prefill_static_workspace, decode_step, gate, lib, library_path,
                  prefill_path, selftest_attention_stall, selftest_bounded_wait,
                  set_profile_events, spec_commit,
                  segmented_workspace_size, spec_verify, static_workspace_status,
                  workspace_size)
from .cache import (PagedCache, cache_attention, cache_attention_shared,  # noqa: F401
                    cache_attention_shared_workspace_size, cache_attention_workspace_size, cache_compact,
                    cache_copy, cache_fork, cache_new, cache_pages_workspace_size, cache_read, cache_resize,
                    cache_write, rotary, rotary_frequencies)

__all__ = ["KDAError", "auto_segments", "chunk_prefill", "chunk_prefill_segmented",
           "segmented_workspace_size", "chunk_prefill_from_host", "chunk_prefill_static_workspace",
           "decode_step", "gate", "lib", "library_path", "prefill_path", "selftest_attention_stall",
           "selftest_bounded_wait",
           "set_profile_events", "spec_commit", "spec_verify", "static_workspace_status",
           "workspace_size", "PagedCache", "cache_attention", "cache_attention_workspace_size",
           "cache_attention_shared", "cache_attention_shared_workspace_size", "cache_compact", "cache_copy", "cache_fork", "cache_new", "cache_pages_workspace_size",
           "cache_read", "cache_resize", "cache_write", "rotary", "rotary_frequencies"]
