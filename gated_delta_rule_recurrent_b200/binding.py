"""ctypes binding of libgdr: torch tensors in, C-ABI calls out.

Only argument marshalling happens here: shape/dtype/device checks (raising
RuntimeError as the op's page specifies in section 异常 of
"lite_boost.ops.recurrent_gated_delta_rule"), the sizes struct, raw device
pointers and the current CUDA stream. Every step of the computation runs in
the library's kernels. Loading fails loudly when libgdr.so is missing; there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

__all__ = ["decode", "decode_gated", "prefill", "prefill_gated", "linear_attention_gate",
           "linear_attention_decode", "linear_attention_prefill", "state_quantize",
           "state_dequantize", "device_error", "GdrError", "lib",
           "library_path", "last_launch", "kernel_forms", "KERNEL_NAMES",
           "STATUS_NAMES", "Dims", "LaunchInfo"]

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))

STATUS_NAMES = {0: "GDR_OK", 1: "GDR_ERR_NULL", 2: "GDR_ERR_DIMS", 3: "GDR_ERR_ALIGN",
                4: "GDR_ERR_UNSUPPORTED", 5: "GDR_ERR_CUDA"}


class GdrError(RuntimeError):
    """A libgdr entry point returned a nonzero status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class Dims(ctypes.Structure):
    """gdr_dims; ``layout`` is 0 (GDR_LAYOUT_KV) unless given."""
    _fields_ = [(n, ctypes.c_int32)
                for n in ("B", "T", "H_qk", "H_v", "D_k", "D_v", "pool_size", "layout")]


class LaunchInfo(ctypes.Structure):
    """gdr_launch_info: one kernel launch (or one kernel form of the dispatcher)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("kernel", "D_k", "tile_cols", "gated", "layout",
                                              "grid", "threads", "smem_bytes", "stages")]

    def as_dict(self) -> dict:
        d = {n: int(getattr(self, n)) for n, _ in self._fields_}
        d["kernel"] = KERNEL_NAMES.get(d["kernel"], d["kernel"])
        d["layout"] = "vk" if d["layout"] == 1 else "kv"
        d["gated"] = bool(d["gated"])
        return d


# gdr_kernel values of include/gdr.h
KERNEL_NAMES = {0: "none", 1: "single_token", 2: "chunked", 3: "tensor_core",
                4: "tensor_core_one", 5: "gate", 6: "prefill", 7: "rows", 8: "linear_decode",
                9: "linear_prefill", 10: "state_cache"}

_P = ctypes.c_void_p
_DECODE_ARGTYPES = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                    ctypes.c_float, _P, _P]
_GATED_ARGTYPES = [ctypes.POINTER(Dims), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                   ctypes.c_float, _P, _P]

_lib = None


def library_path() -> str:
    return os.environ.get("GDR_LIBRARY", os.path.join(_PKG_DIR, "libgdr.so"))


def lib() -> ctypes.CDLL:
    """The loaded libgdr.so (loaded once; raises if it is missing)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"libgdr.so not found at {path}; build it with "
                "`python -m gated_delta_rule_recurrent_b200.build`")
        L = ctypes.CDLL(path)
        L.gdr_decode.argtypes = _DECODE_ARGTYPES
        L.gdr_decode.restype = ctypes.c_int
        L.gdr_gate_fused.argtypes = _GATED_ARGTYPES
        L.gdr_gate_fused.restype = ctypes.c_int
        L.gdr_prefill.argtypes = _DECODE_ARGTYPES
        L.gdr_prefill.restype = ctypes.c_int
        L.gdr_prefill_gated.argtypes = _GATED_ARGTYPES
        L.gdr_prefill_gated.restype = ctypes.c_int
        L.gdr_status_string.argtypes = [ctypes.c_int]
        L.gdr_status_string.restype = ctypes.c_char_p
        L.gdr_last_error.argtypes = []
        L.gdr_last_error.restype = ctypes.c_char_p
        L.gdr_abi_version.argtypes = []
        L.gdr_abi_version.restype = ctypes.c_int
        L.gdr_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
        L.gdr_device_error.restype = ctypes.c_int
        P = ctypes.c_void_p
        L.gdr_linear_attention_gate.argtypes = [P, P, P, P, P, P, ctypes.c_int64, ctypes.c_int32,
                                                ctypes.c_int, P]
        L.gdr_linear_attention_gate.restype = ctypes.c_int
        D, I = ctypes.POINTER(Dims), ctypes.c_int32
        L.gdr_linear_attention_decode.argtypes = [D, P, P, P, P, P, P, P, P, ctypes.c_float, P, P]
        L.gdr_linear_attention_decode.restype = ctypes.c_int
        L.gdr_linear_attention_prefill.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_float, P, P,
                                                   ctypes.c_int64, P]
        L.gdr_linear_attention_prefill.restype = ctypes.c_int
        L.gdr_linear_attention_prefill_workspace.argtypes = [D, ctypes.POINTER(ctypes.c_int64)]
        L.gdr_linear_attention_prefill_workspace.restype = ctypes.c_int
        L.gdr_state_quantize.argtypes = [P, I, P, P, P, I, P, I, ctypes.c_int64, ctypes.c_int, P]
        L.gdr_state_quantize.restype = ctypes.c_int
        L.gdr_state_dequantize.argtypes = [P, P, I, P, P, I, P, I, ctypes.c_int64, ctypes.c_int,
                                           P]
        L.gdr_state_dequantize.restype = ctypes.c_int
        L.gdr_last_launch.argtypes = [ctypes.POINTER(LaunchInfo)]
        L.gdr_last_launch.restype = ctypes.c_int
        L.gdr_kernel_form_count.argtypes = []
        L.gdr_kernel_form_count.restype = ctypes.c_int
        L.gdr_kernel_form.argtypes = [ctypes.c_int, ctypes.POINTER(LaunchInfo)]
        L.gdr_kernel_form.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != 0:
        raise GdrError(rc, lib().gdr_last_error().decode())


def device_error(reset: bool = True, device=None) -> int:
    """The device error word of ``device`` (bit 0: a consumer wait ran out of time,
    bit 1: a producer wait, bit 2: the final drain). Synchronises the device."""
    flags = ctypes.c_uint32(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        rc = lib().gdr_device_error(ctypes.byref(flags), int(bool(reset)))
    _check(rc)
    return int(flags.value)


def last_launch() -> dict:
    """The calling thread's most recent kernel launch through the library
    (``gdr_last_launch``): kernel family, D_k, tile columns, gate, layout and
    the launch shape. ``kernel`` is "none" after a call that queued nothing."""
    info = LaunchInfo()
    _check(lib().gdr_last_launch(ctypes.byref(info)))
    return info.as_dict()


def kernel_forms() -> list:
    """Every gated-delta-rule kernel form the dispatcher can choose (``gdr_kernel_form``),
    as dicts with kernel, D_k, tile_cols, gated and layout. Needs no GPU."""
    L = lib()
    forms = []
    for i in range(L.gdr_kernel_form_count()):
        info = LaunchInfo()
        _check(L.gdr_kernel_form(i, ctypes.byref(info)))
        d = info.as_dict()
        forms.append({k: d[k] for k in ("kernel", "D_k", "tile_cols", "gated", "layout")})
    return forms


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise RuntimeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise RuntimeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise RuntimeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise RuntimeError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# gdr_state_layout values of include/gdr.h
_LAYOUTS = {"kv": 0, "vk": 1}


def _common(query, key, value, state_pool, actual_seq_lengths, ssm_state_indices, gk,
            num_accepted_tokens, out, state_layout="kv"):
    if not isinstance(query, torch.Tensor) or query.dim() != 4:
        raise RuntimeError("query must be a 4-D tensor [B, H_qk, T, D_k]")
    device = query.device
    if device.type != "cuda":
        raise RuntimeError("all tensors must be on a CUDA device")
    B, H_qk, T, D_k = query.shape
    if not isinstance(value, torch.Tensor) or value.dim() != 4:
        raise RuntimeError("value must be a 4-D tensor [B, H_v, T, D_v]")
    H_v, D_v = value.shape[1], value.shape[3]
    if state_layout not in _LAYOUTS:
        raise RuntimeError('state_layout must be "kv" ([pool, H_v, D_k, D_v]) or "vk" '
                           '([pool, H_v, D_v, D_k])')
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 4:
        raise RuntimeError("state_pool must be a 4-D tensor [pool, H_v, D_k, D_v] "
                           "(or [pool, H_v, D_v, D_k] for state_layout='vk')")
    P = state_pool.shape[0]
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    _need(query, "query", bf16, (B, H_qk, T, D_k), device)
    _need(key, "key", bf16, (B, H_qk, T, D_k), device)
    _need(value, "value", bf16, (B, H_v, T, D_v), device)
    _need(state_pool, "state_pool", bf16,
          (P, H_v, D_k, D_v) if state_layout == "kv" else (P, H_v, D_v, D_k), device)
    _need(actual_seq_lengths, "actual_seq_lengths", i32, (B,), device)
    _need(ssm_state_indices, "ssm_state_indices", i32, (B,), device)
    _need(gk, "gk", f32, (B, H_v, T, D_k), device)
    if num_accepted_tokens is not None:
        _need(num_accepted_tokens, "num_accepted_tokens", i32, (B,), device)
    if out is None:
        out = torch.empty((B, H_v, T, D_v), dtype=bf16, device=device)
    else:
        _need(out, "out", bf16, (B, H_v, T, D_v), device)
    dims = Dims(B, T, H_qk, H_v, D_k, D_v, P, _LAYOUTS[state_layout])
    stream = ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    return device, dims, out, stream


def decode(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, beta: torch.Tensor,
           state_pool: torch.Tensor, actual_seq_lengths: torch.Tensor,
           ssm_state_indices: torch.Tensor, g: torch.Tensor, gk: torch.Tensor,
           num_accepted_tokens: Optional[torch.Tensor] = None, scale_value: float = 1.0, *,
           out: Optional[torch.Tensor] = None,
           state_layout: str = "kv") -> Tuple[torch.Tensor, torch.Tensor]:
    """recurrent_gated_delta_rule decode step through ``gdr_decode``.

    Argument order and defaults follow the op's page. ``state_pool`` is
    updated in place and returned as the second result (the page's
    ``state_out``). ``num_accepted_tokens`` (optional, [B] int32) is the
    number of leading tokens whose state update is committed: outputs of all
    valid tokens are computed, the slot keeps the state after the first n
    (unchanged for n = 0); None commits them all. ``state_layout`` "vk" takes
    the pool as [pool, H_v, D_v, D_k] (k contiguous) instead of the page's
    [pool, H_v, D_k, D_v]. Queued on the current CUDA stream; no
    synchronisation.
    """
    device, dims, out, stream = _common(query, key, value, state_pool, actual_seq_lengths,
                                        ssm_state_indices, gk, num_accepted_tokens, out,
                                        state_layout)
    B, H_v, T = dims.B, dims.H_v, dims.T
    _need(beta, "beta", torch.bfloat16, (B, H_v, T), device)
    _need(g, "g", torch.float32, (B, H_v, T), device)
    with torch.cuda.device(device):
        rc = lib().gdr_decode(ctypes.byref(dims), _ptr(query), _ptr(key), _ptr(value),
                              _ptr(beta), _ptr(state_pool), _ptr(actual_seq_lengths),
                              _ptr(ssm_state_indices), _ptr(g), _ptr(gk),
                              _ptr(num_accepted_tokens), float(scale_value), _ptr(out), stream)
    _check(rc)
    return out, state_pool


def decode_gated(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, a: torch.Tensor,
                 b: torch.Tensor, dt_bias: torch.Tensor, decay_scale: torch.Tensor,
                 state_pool: torch.Tensor, actual_seq_lengths: torch.Tensor,
                 ssm_state_indices: torch.Tensor, gk: torch.Tensor,
                 num_accepted_tokens: Optional[torch.Tensor] = None, scale_value: float = 1.0,
                 *, out: Optional[torch.Tensor] = None,
                 state_layout: str = "kv") -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode step with the LinearAttentionGate prologue fused, through ``gdr_gate_fused``.

    ``a`` and ``b`` are [B, T, H_v] bf16; ``dt_bias`` and ``decay_scale`` are
    [H_v] fp32. g and beta are computed inside the kernel. ``state_layout`` as
    for ``decode``.
    """
    device, dims, out, stream = _common(query, key, value, state_pool, actual_seq_lengths,
                                        ssm_state_indices, gk, num_accepted_tokens, out,
                                        state_layout)
    B, H_v, T = dims.B, dims.H_v, dims.T
    _need(a, "a", torch.bfloat16, (B, T, H_v), device)
    _need(b, "b", torch.bfloat16, (B, T, H_v), device)
    _need(dt_bias, "dt_bias", torch.float32, (H_v,), device)
    _need(decay_scale, "decay_scale", torch.float32, (H_v,), device)
    with torch.cuda.device(device):
        rc = lib().gdr_gate_fused(ctypes.byref(dims), _ptr(query), _ptr(key), _ptr(value),
                                  _ptr(a), _ptr(b), _ptr(dt_bias), _ptr(decay_scale),
                                  _ptr(state_pool), _ptr(actual_seq_lengths),
                                  _ptr(ssm_state_indices), _ptr(gk),
                                  _ptr(num_accepted_tokens), float(scale_value), _ptr(out),
                                  stream)
    _check(rc)
    return out, state_pool


def prefill(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, beta: torch.Tensor,
            state_pool: torch.Tensor, actual_seq_lengths: torch.Tensor,
            ssm_state_indices: torch.Tensor, g: torch.Tensor, gk: torch.Tensor,
            num_accepted_tokens: Optional[torch.Tensor] = None, scale_value: float = 1.0, *,
            out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The recurrence over a long prompt through ``gdr_prefill``: the arguments
    and results of ``decode`` for any token count T (D_k = 128, D_v a multiple
    of 128, the [pool, H_v, D_k, D_v] pool)."""
    device, dims, out, stream = _common(query, key, value, state_pool, actual_seq_lengths,
                                        ssm_state_indices, gk, num_accepted_tokens, out, "kv")
    B, H_v, T = dims.B, dims.H_v, dims.T
    _need(beta, "beta", torch.bfloat16, (B, H_v, T), device)
    _need(g, "g", torch.float32, (B, H_v, T), device)
    with torch.cuda.device(device):
        rc = lib().gdr_prefill(ctypes.byref(dims), _ptr(query), _ptr(key), _ptr(value),
                               _ptr(beta), _ptr(state_pool), _ptr(actual_seq_lengths),
                               _ptr(ssm_state_indices), _ptr(g), _ptr(gk),
                               _ptr(num_accepted_tokens), float(scale_value), _ptr(out), stream)
    _check(rc)
    return out, state_pool


def prefill_gated(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, a: torch.Tensor,
                  b: torch.Tensor, dt_bias: torch.Tensor, decay_scale: torch.Tensor,
                  state_pool: torch.Tensor, actual_seq_lengths: torch.Tensor,
                  ssm_state_indices: torch.Tensor, gk: torch.Tensor,
                  num_accepted_tokens: Optional[torch.Tensor] = None, scale_value: float = 1.0,
                  *, out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``prefill`` with the LinearAttentionGate fused, through ``gdr_prefill_gated``
    (the gate arguments of ``decode_gated``)."""
    device, dims, out, stream = _common(query, key, value, state_pool, actual_seq_lengths,
                                        ssm_state_indices, gk, num_accepted_tokens, out, "kv")
    B, H_v, T = dims.B, dims.H_v, dims.T
    _need(a, "a", torch.bfloat16, (B, T, H_v), device)
    _need(b, "b", torch.bfloat16, (B, T, H_v), device)
    _need(dt_bias, "dt_bias", torch.float32, (H_v,), device)
    _need(decay_scale, "decay_scale", torch.float32, (H_v,), device)
    with torch.cuda.device(device):
        rc = lib().gdr_prefill_gated(ctypes.byref(dims), _ptr(query), _ptr(key), _ptr(value),
                                     _ptr(a), _ptr(b), _ptr(dt_bias), _ptr(decay_scale),
                                     _ptr(state_pool), _ptr(actual_seq_lengths),
                                     _ptr(ssm_state_indices), _ptr(gk),
                                     _ptr(num_accepted_tokens), float(scale_value), _ptr(out),
                                     stream)
    _check(rc)
    return out, state_pool


# gdr_dtype values of include/gdr.h
_GATE_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def linear_attention_gate(a: torch.Tensor, dt_bias: torch.Tensor, decay_scale: torch.Tensor,
                          b: Optional[torch.Tensor] = None, want_beta: Optional[bool] = None,
                          decay: Optional[torch.Tensor] = None,
                          beta: Optional[torch.Tensor] = None):
    """The LinearAttentionGate op on its own ("com.microsoft.LinearAttentionGate").

    decay = decay_scale * softplus(a + dt_bias) and, when requested, beta =
    sigmoid(b), computed in float32 and narrowed to a's dtype (float32, float16
    or bfloat16). The head axis is the last axis of ``a``; dt_bias and
    decay_scale are float32 [H]. ``want_beta`` defaults to ``b is not None``;
    requesting beta without b is an error (the page's rule), while a b given
    with want_beta=False is accepted and not read. Returns (decay, beta or None).
    """
    if not isinstance(a, torch.Tensor) or a.dim() < 1:
        raise RuntimeError("a must be a tensor of rank >= 1 (heads on the last axis)")
    device = a.device
    if device.type != "cuda":
        raise RuntimeError("all tensors must be on a CUDA device")
    if a.dtype not in _GATE_DTYPES:
        raise RuntimeError(f"a must be float32, float16 or bfloat16, got {a.dtype}")
    if want_beta is None:
        want_beta = b is not None
    if want_beta and b is None:
        raise RuntimeError("beta was requested but b is None")
    H = a.shape[-1]
    _need(a, "a", a.dtype, a.shape, device)
    _need(dt_bias, "dt_bias", torch.float32, (H,), device)
    _need(decay_scale, "decay_scale", torch.float32, (H,), device)
    if b is not None:
        _need(b, "b", a.dtype, a.shape, device)
    if decay is None:
        decay = torch.empty_like(a)
    _need(decay, "decay", a.dtype, a.shape, device)
    if want_beta:
        if beta is None:
            beta = torch.empty_like(a)
        _need(beta, "beta", a.dtype, a.shape, device)
    else:
        beta = None
    rows = a.numel() // H if H > 0 else 0
    stream = torch.cuda.current_stream(device).cuda_stream
    with torch.cuda.device(device):
        rc = lib().gdr_linear_attention_gate(
            _ptr(a), _ptr(b if want_beta else None), _ptr(dt_bias), _ptr(decay_scale),
            _ptr(decay), _ptr(beta), rows, H, _GATE_DTYPES[a.dtype], ctypes.c_void_p(stream))
    _check(rc)
    return decay, beta


def _call(index: int, fn, *args) -> None:
    """The library's ``fn(*args)`` with CUDA device ``index`` as the current one."""
    if _device() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != 0:
        _check(rc)


# The current device, without the check for initialisation around it (a CUDA
# tensor is there) where this torch has the function.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# The handle of a device's current stream, without the Stream object around it
# where this torch has the function.
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _linear_args(query, key, value, log_decay, state_pool, actual_seq_lengths,
                 ssm_state_indices, num_accepted_tokens, out):
    """(device index, Dims, out) of a linear-attention call, its tensors checked."""
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    try:
        index = query.get_device()
        B, H_qk, T, D_k = qk = query.shape
        _, H_v, _, D_v = value.shape
        P = state_pool.shape[0]
        # every condition of the list below, in one go: a call costs a few
        # microseconds of the host, and a step of one sequence no more of the GPU
        good = (
            index >= 0 and query.dtype is bf16 and key.dtype is bf16 and value.dtype is bf16
            and state_pool.dtype is bf16 and log_decay.dtype is f32
            and actual_seq_lengths.dtype is i32 and ssm_state_indices.dtype is i32
            and key.shape == qk and value.shape == (B, H_v, T, D_v)
            and state_pool.shape == (P, H_v, D_k, D_v) and log_decay.shape == (H_v,)
            and actual_seq_lengths.shape == (B,) and ssm_state_indices.shape == (B,)
            and key.get_device() == index and value.get_device() == index
            and state_pool.get_device() == index and log_decay.get_device() == index
            and actual_seq_lengths.get_device() == index
            and ssm_state_indices.get_device() == index
            and query.is_contiguous() and key.is_contiguous() and value.is_contiguous()
            and state_pool.is_contiguous() and log_decay.is_contiguous()
            and actual_seq_lengths.is_contiguous() and ssm_state_indices.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        good = False
    if not good:  # which one
        for t, name, dims in ((query, "query", "[B, H_qk, T, D_k]"),
                              (value, "value", "[B, H_v, T, D_v]"),
                              (state_pool, "state_pool", "[pool, H_v, D_k, D_v]")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise RuntimeError(f"{name} must be a 4-D tensor {dims}")
        if not query.is_cuda:
            raise RuntimeError("all tensors must be on a CUDA device")
        B, H_qk, T, D_k = qk = tuple(query.shape)
        H_v, D_v, P = value.shape[1], value.shape[3], state_pool.shape[0]
        for t, name, dtype, shape in (
                (query, "query", bf16, qk), (key, "key", bf16, qk),
                (value, "value", bf16, (B, H_v, T, D_v)), (log_decay, "log_decay", f32, (H_v,)),
                (state_pool, "state_pool", bf16, (P, H_v, D_k, D_v)),
                (actual_seq_lengths, "actual_seq_lengths", i32, (B,)),
                (ssm_state_indices, "ssm_state_indices", i32, (B,))):
            _need(t, name, dtype, shape, query.device)
    if num_accepted_tokens is not None:
        _need(num_accepted_tokens, "num_accepted_tokens", i32, (B,), query.device)
    if out is None:
        out = torch.empty_like(value)
    else:
        _need(out, "out", bf16, value.shape, query.device)
    return index, Dims(B, T, H_qk, H_v, D_k, D_v, P), out


def linear_attention_decode(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                            log_decay: torch.Tensor, state_pool: torch.Tensor,
                            actual_seq_lengths: torch.Tensor, ssm_state_indices: torch.Tensor,
                            num_accepted_tokens: Optional[torch.Tensor] = None,
                            scale_value: float = 1.0, *,
                            out: Optional[torch.Tensor] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Linear attention with one decay per head for one to eight tokens, through
    ``gdr_linear_attention_decode``: S = S * exp(log_decay[h]) + k v^T, then
    o = S^T (q * scale_value), token by token.

    ``log_decay`` is [H_v] float32; every other argument, and the in-place
    update of ``state_pool`` (the second result), as for ``decode``. Queued on
    the current CUDA stream; no synchronisation.
    """
    index, dims, out = _linear_args(query, key, value, log_decay, state_pool,
                                    actual_seq_lengths, ssm_state_indices,
                                    num_accepted_tokens, out)
    accepted = None if num_accepted_tokens is None else num_accepted_tokens.data_ptr()
    _call(index, lib().gdr_linear_attention_decode, ctypes.byref(dims), query.data_ptr(),
          key.data_ptr(), value.data_ptr(), log_decay.data_ptr(), state_pool.data_ptr(),
          actual_seq_lengths.data_ptr(), ssm_state_indices.data_ptr(), accepted,
          float(scale_value), out.data_ptr(), _stream(index))
    return out, state_pool


def linear_attention_prefill(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                             log_decay: torch.Tensor, state_pool: torch.Tensor,
                             actual_seq_lengths: torch.Tensor, ssm_state_indices: torch.Tensor,
                             scale_value: float = 1.0, *, out: Optional[torch.Tensor] = None
                             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The recurrence of ``linear_attention_decode`` over prompts of any length,
    through ``gdr_linear_attention_prefill`` (chunks of 128 tokens on the tensor
    cores). All valid tokens are committed. An infinity or NaN in a valid token's
    value may reach its column of the outputs of the tokens before it in its chunk.
    Queued on the current CUDA stream; no synchronisation.
    """
    index, dims, out = _linear_args(query, key, value, log_decay, state_pool,
                                    actual_seq_lengths, ssm_state_indices, None, out)
    L = lib()
    need = ctypes.c_int64(0)
    _call(index, L.gdr_linear_attention_prefill_workspace, ctypes.byref(dims),
          ctypes.byref(need))
    # a workspace of this call's own: the allocator gives it to no other stream
    # or graph while the call runs
    size, work, at = need.value, None, None
    if size:
        work = torch.empty(size, dtype=torch.uint8, device=query.device)
        at = work.data_ptr()
    _call(index, L.gdr_linear_attention_prefill, ctypes.byref(dims), query.data_ptr(),
          key.data_ptr(), value.data_ptr(), log_decay.data_ptr(), state_pool.data_ptr(),
          actual_seq_lengths.data_ptr(), ssm_state_indices.data_ptr(), float(scale_value),
          out.data_ptr(), at, size, _stream(index))
    return out, state_pool


# gdr_cache_type values of include/gdr.h
_CACHE_TYPES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_CACHE_GROUP = 64


def _cache_args(state_pool, ssm_state_indices, cache, scales, cache_indices):
    """(device index, slots, entries, pairs, values of a slot, cache type) of a cache call,
    its tensors checked."""
    i32 = torch.int32
    try:
        index = state_pool.get_device()
        P, H, R, C = state_pool.shape
        N = cache.shape[0]
        n, = ssm_state_indices.shape
        kind = _CACHE_TYPES.get(cache.dtype)
        good = (  # in one go, as in _linear_args
            index >= 0 and kind is not None and C % _CACHE_GROUP == 0
            and state_pool.dtype is torch.bfloat16 and scales.dtype is torch.float32
            and ssm_state_indices.dtype is i32 and cache_indices.dtype is i32
            and cache.shape == (N, H, R, C) and scales.shape == (N, H, R, C // _CACHE_GROUP)
            and cache_indices.shape == (n,) and cache.get_device() == index
            and scales.get_device() == index and ssm_state_indices.get_device() == index
            and cache_indices.get_device() == index and state_pool.is_contiguous()
            and cache.is_contiguous() and scales.is_contiguous()
            and ssm_state_indices.is_contiguous() and cache_indices.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        good = False
    if not good:  # which one
        for t, name in ((state_pool, "state_pool"), (cache, "cache")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise RuntimeError(f"{name} must be a 4-D tensor ([pool or entries, H_v, rows, "
                                   "columns])")
        if not state_pool.is_cuda:
            raise RuntimeError("all tensors must be on a CUDA device")
        if cache.dtype not in _CACHE_TYPES:
            raise RuntimeError(f"cache must be int8 or float8_e4m3fn, got {cache.dtype}")
        P, H, R, C = state_pool.shape
        N = cache.shape[0]
        if C % _CACHE_GROUP != 0:
            raise RuntimeError("state_pool's last axis must be a multiple of 64")
        if not isinstance(ssm_state_indices, torch.Tensor) or ssm_state_indices.dim() != 1:
            raise RuntimeError("ssm_state_indices must be a 1-D tensor")
        n = ssm_state_indices.shape[0]
        for t, name, dtype, shape in (
                (state_pool, "state_pool", torch.bfloat16, (P, H, R, C)),
                (cache, "cache", cache.dtype, (N, H, R, C)),
                (scales, "scales", torch.float32, (N, H, R, C // _CACHE_GROUP)),
                (ssm_state_indices, "ssm_state_indices", i32, (n,)),
                (cache_indices, "cache_indices", i32, (n,))):
            _need(t, name, dtype, shape, state_pool.device)
    return index, P, N, n, H * R * C, kind


def state_quantize(state_pool: torch.Tensor, ssm_state_indices: torch.Tensor,
                   cache: torch.Tensor, scales: torch.Tensor, cache_indices: torch.Tensor
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Write slots of a state pool to an 8-bit cache through ``gdr_state_quantize``:
    slot ``ssm_state_indices[i]`` to entry ``cache_indices[i]`` (both [n] int32,
    entries distinct; a pair outside its range is skipped).

    ``state_pool`` is [pool, H_v, D_k, D_v] or [pool, H_v, D_v, D_k] bfloat16,
    ``cache`` [entries, ...] of the same slot shape in int8 or float8_e4m3fn,
    ``scales`` [entries, H_v, rows, columns / 64] float32: 64 consecutive
    values share a scale. Returns (cache, scales). Queued on the current CUDA
    stream; no synchronisation.
    """
    index, P, N, n, values, kind = _cache_args(state_pool, ssm_state_indices, cache, scales,
                                               cache_indices)
    _call(index, lib().gdr_state_quantize, state_pool.data_ptr(), P,
          ssm_state_indices.data_ptr(), cache.data_ptr(), scales.data_ptr(), N,
          cache_indices.data_ptr(), n, values, kind, _stream(index))
    return cache, scales


def state_dequantize(cache: torch.Tensor, scales: torch.Tensor, cache_indices: torch.Tensor,
                     state_pool: torch.Tensor, ssm_state_indices: torch.Tensor) -> torch.Tensor:
    """Read entries of an 8-bit cache back into slots of a state pool through
    ``gdr_state_dequantize``: entry ``cache_indices[i]`` to slot
    ``ssm_state_indices[i]`` (slots distinct; one entry may go to several slots).
    The tensors are those of ``state_quantize``. Returns ``state_pool``, updated
    in place. Queued on the current CUDA stream; no synchronisation.
    """
    index, P, N, n, values, kind = _cache_args(state_pool, ssm_state_indices, cache, scales,
                                               cache_indices)
    _call(index, lib().gdr_state_dequantize, cache.data_ptr(), scales.data_ptr(), N,
          cache_indices.data_ptr(), state_pool.data_ptr(), P, ssm_state_indices.data_ptr(), n,
          values, kind, _stream(index))
    return state_pool
