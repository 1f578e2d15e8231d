"""Exact attention forward (bf16 and FP8 inputs), backward, paged-KV decoding (bf16 and 8-bit
caches), the paged cache's append and ring attention across GPUs for NVIDIA B200 (sm_100a).

``fwd``, ``fwd_fp8``, ``bwd``, ``decode``, ``decode_kv8`` and ``kv_append`` (and ``fwd_host`` /
``fwd_fp8_host`` on host tensors, with the copies overlapped) run the hand-written
kernels of ``libattn_b200.so`` through its C ABI (include/attn.h); there is no CPU or
library fallback.
"""
from .attn import (AttnError, MASKS, bwd, bwd_debug_error, debug_error, decode, decode_debug_error,  # noqa: F401
                   decode_kv8, decode_kv8_debug_error, decode_kv8_num_splits, decode_kv8_workspace,
                   decode_kv8_workspace_bytes, decode_num_splits, decode_static, decode_workspace_bytes, fwd, fwd_fp8,
                   fwd_fp8_host, fwd_host, kv_append, kv_append_debug_error, load_library, merge, num_work_items)
from . import ring  # noqa: F401

__all__ = ["fwd", "fwd_fp8", "fwd_host", "fwd_fp8_host", "bwd", "bwd_debug_error", "decode", "decode_debug_error",
           "decode_kv8", "decode_kv8_debug_error", "decode_kv8_num_splits", "decode_kv8_workspace",
           "decode_kv8_workspace_bytes", "decode_num_splits", "decode_static", "decode_workspace_bytes", "debug_error",
           "kv_append", "kv_append_debug_error", "load_library", "merge", "num_work_items", "ring", "AttnError", "MASKS"]
