"""Recurrent gated-delta-rule decode step (and long-prompt prefill) for B200 (sm_100a),
linear attention with one decay per head on the same state pool, and the pool's 8-bit cache.

The compute path is the C-ABI library ``libgdr.so`` built from ``csrc/``; the
Python functions here only marshal torch tensors into it. Importing the
package does not load the library: the first use of ``decode``,
``decode_gated``, ``prefill``, ``prefill_gated``, ``linear_attention_gate``,
``linear_attention_decode``, ``linear_attention_prefill``, ``state_quantize``,
``state_dequantize`` or ``lib`` does, and raises if it is missing (there is no CPU fallback).
"""
from __future__ import annotations

__all__ = ["decode", "decode_gated", "prefill", "prefill_gated", "linear_attention_gate",
           "linear_attention_decode", "linear_attention_prefill", "state_quantize",
           "state_dequantize", "device_error", "GdrError", "lib", "library_path", "last_launch",
           "kernel_forms"]

_LAZY = {"decode", "decode_gated", "prefill", "prefill_gated", "linear_attention_gate",
         "linear_attention_decode", "linear_attention_prefill", "state_quantize",
         "state_dequantize", "device_error", "GdrError", "lib", "library_path", "STATUS_NAMES",
         "last_launch", "kernel_forms"}


_binding = None  # the module behind the names, once it is loaded


def __getattr__(name):
    global _binding
    if name in _LAZY:
        if _binding is None:
            from . import binding as _binding
        return getattr(_binding, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
