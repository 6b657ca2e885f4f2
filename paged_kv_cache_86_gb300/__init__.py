"""Attention over a block-paged KV cache on one GB300 GPU.

The compute path is the C-ABI library ``libpkv.so`` (hand-written sm_103a
CUDA kernels, declared in ``include/pkv.h``); this package is its thin ctypes
binding plus the seeded synthetic workload generator used by tests and the
bench. Importing the package does not load the library; the first call does,
and fails loudly if it has not been built.
"""
from ._lib import (PkvError, SlotPlan, copy_blocks, decode_step, decode_step_fp8,
                   decode_window_workspace_size, decode_workspace_size, get_device_errors, load,
                   load_kvcache_fp8_block, mixed_step, mixed_workspace_size, paged_decode,
                   paged_decode_fp8, paged_decode_fp8_block, paged_decode_window, paged_prefill,
                   paged_prefill_window, plan_slots, prefill_workspace_size, qk_norm_rope,
                   qk_norm_rope_store, selftest_bounded_wait, store_kvcache, store_kvcache_fp8,
                   store_kvcache_fp8_block, tree_decode, tree_decode_workspace_size, tree_masks,
                   version)

__all__ = ["PkvError", "SlotPlan", "copy_blocks", "decode_step", "decode_step_fp8",
           "decode_window_workspace_size", "decode_workspace_size", "get_device_errors", "load",
           "load_kvcache_fp8_block", "mixed_step", "mixed_workspace_size", "paged_decode",
           "paged_decode_fp8", "paged_decode_fp8_block", "paged_decode_window", "paged_prefill",
           "paged_prefill_window", "plan_slots", "prefill_workspace_size", "qk_norm_rope",
           "qk_norm_rope_store", "selftest_bounded_wait", "store_kvcache", "store_kvcache_fp8",
           "store_kvcache_fp8_block", "tree_decode", "tree_decode_workspace_size", "tree_masks",
           "version"]
