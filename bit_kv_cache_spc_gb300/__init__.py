"""Python binding of libspc, the GB300 decode-time hot path of SpeCache.

Every ``spc_*`` function here has the name and arguments of the C entry point
in ``include/spc.h`` and only marshals arguments: torch tensors become device
pointers, the stream defaults to torch's current stream, and a non-OK status
raises ``SpcError``.  All computation runs in the CUDA kernels of
``libspc.so``; there is no other implementation behind these names.  If the
library has not been built the import fails: build it with
``python -c "import __graft_entry__ as g; g.build()"``.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
import os
import struct

import torch

__all__ = [
    "Dims", "SpcError", "spc_abi_version", "spc_num_quantized", "spc_records_bytes", "spc_resid_bytes",
    "spc_quantize_kv", "spc_attn_workspace_bytes", "spc_decode_attn2", "spc_merged_attn", "spc_topk_select",
    "spc_topk_select_prev", "spc_merged_attn_fetch_prev", "spc_host_gather_prev", "spc_decode_step_prev",
    "spc_host_gather", "spc_merged_attn_noalloc", "spc_merged_attn_fetch", "spc_attn_kernel_count",
    "spc_decode_step_kernel_count", "spc_decode_step_on_chip", "spc_decode_step", "spc_step_workspace_bytes",
    "spc_read_device_status", "spc_append_kv", "spc_offload_kv", "spc_rope_frequencies", "spc_rope",
    "spc_rope_axes", "spc_norm_rope",
    "spc_prompt_attn", "spc_prompt_attn_workspace_bytes", "spc_prompt_attn_status",
    "spc_prompt_attn_wait_limit", "spc_window_attn", "spc_window_attn_workspace_bytes", "spc_prefix_attn",
    "spc_prefix_attn_workspace_bytes", "spc_prefix_attn_together", "spc_extend_kv", "spc_dequantize_kv", "lib_path",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libspc.so")

if not os.path.exists(lib_path):
    raise ImportError(f"{lib_path} is missing: the CUDA library must be built (see __graft_entry__.build())")
_lib = C.CDLL(lib_path)

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "CUDA error",
          4: "host pointer is not mapped pinned memory", 5: "workspace too small",
          6: "a kernel's bounded wait ran out"}


class SpcError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = f"{fn}: {STATUS.get(status, status)}"
        if status == 3:
            msg += f" (cudaError {_lib.spc_last_cuda_error()})"
        super().__init__(msg)


class spc_dims(C.Structure):
    _fields_ = [("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("D", C.c_int32),
                ("bits", C.c_int32), ("group", C.c_int32), ("N", C.c_int32), ("R", C.c_int32),
                ("q_groups_cap", C.c_int32), ("resid_cap", C.c_int32), ("scale", C.c_float)]


def Dims(B, Hq, Hkv, N, R, bits, q_groups_cap=None, resid_cap=None, scale=None, D=128, group=32) -> spc_dims:
    """Shape of one layer's cache (see spc_dims in include/spc.h).  The default
    capacities hold exactly the N_q quantised tokens and the r = N - N_q
    residual rows that spc_num_quantized reports for the shape."""
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if q_groups_cap is None or resid_cap is None:
        probe = spc_dims(B, Hq, Hkv, D, bits, group, N, R, max(N, 0) // 32 + 1, max(N, 0), scale)
        nq = max(int(_lib.spc_num_quantized(C.byref(probe))), 0)  # -1: an invalid shape, which every call refuses
        if q_groups_cap is None:
            q_groups_cap = nq // 32
        if resid_cap is None:
            resid_cap = N - nq
    return spc_dims(B, Hq, Hkv, D, bits, group, N, R, q_groups_cap, resid_cap, scale)


class spc_layout(C.Structure):
    _fields_ = [("b", C.c_int64), ("t", C.c_int64), ("h", C.c_int64)]


class spc_rope_scaling(C.Structure):
    _fields_ = [("kind", C.c_int32), ("theta", C.c_double), ("factor", C.c_double), ("low", C.c_double),
                ("high", C.c_double), ("context", C.c_double)]


class spc_rope_dims(C.Structure):
    _fields_ = [("B", C.c_int32), ("T", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("D", C.c_int32),
                ("rot", C.c_int32), ("interleaved", C.c_int32), ("mscale", C.c_float)] + [
                    (n, spc_layout) for n in ("q", "k", "v", "q_out", "k_out", "v_out")]


class spc_norm_rope_dims(C.Structure):
    _fields_ = [("rope", spc_rope_dims), ("axes", C.c_int32), ("eps", C.c_float), ("axis", C.c_uint8 * 64)]


class spc_prompt_dims(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("S", "Hq", "Hkv", "D", "q_tokens", "k_tokens", "q_max", "k_max")] + [
        ("scale", C.c_float)] + [(n, spc_layout) for n in ("q", "k", "v", "o")]


class spc_prefix(C.Structure):
    _fields_ = [("tokens", C.c_int32), ("k", spc_layout), ("v", spc_layout)]


_P = C.c_void_p
_D = C.POINTER(spc_dims)
_sig = {
    "spc_abi_version": (C.c_int32, []),
    "spc_status_string": (C.c_char_p, [C.c_int]),
    "spc_last_cuda_error": (C.c_int32, []),
    "spc_num_quantized": (C.c_int32, [_D]),
    "spc_records_bytes": (C.c_size_t, [_D]),
    "spc_resid_bytes": (C.c_size_t, [_D]),
    "spc_quantize_kv": (C.c_int, [_D, _P, _P, _P, _P, _P]),
    "spc_attn_workspace_bytes": (C.c_size_t, [_D, C.c_int32]),
    "spc_decode_attn2": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "spc_merged_attn": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, C.c_int32, _P, _P, _P, _P, C.c_size_t, _P]),
    "spc_merged_attn_noalloc": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, C.c_int32, _P, _P, _P, _P]),
    "spc_merged_attn_fetch": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, C.c_int32, _P, _P, _P, _P, C.c_size_t,
                                        _P, C.c_int64, _P, C.c_int32, _P, _P]),
    "spc_topk_select": (C.c_int, [_D, _P, _P, C.c_int32, _P, _P, _P]),
    "spc_topk_select_prev": (C.c_int, [_D, _P, _P, C.c_int32, _P, _P, _P, C.c_int32, _P, _P]),
    "spc_merged_attn_fetch_prev": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, C.c_int32, _P, _P, _P, _P, C.c_size_t,
                                             _P, C.c_int64, _P, C.c_int32, _P, _P, _P, C.c_int32, _P]),
    "spc_host_gather": (C.c_int, [_D, _P, C.c_int64, _P, C.c_int32, _P, C.c_int32, _P]),
    "spc_host_gather_prev": (C.c_int, [_D, _P, C.c_int64, _P, C.c_int32, _P, _P, _P, C.c_int32, C.c_int32, _P]),
    "spc_append_kv": (C.c_int, [_D, _P, _P, _P, _P, _P, C.c_int64, _P]),
    "spc_offload_kv": (C.c_int, [_D, _P, _P, _P, C.c_int64, _P]),
    "spc_step_workspace_bytes": (C.c_size_t, [_D, C.c_int32]),
    "spc_attn_kernel_count": (C.c_int32, [_D, C.c_int32, C.c_int32]),
    "spc_decode_step_kernel_count": (C.c_int32, [_D, C.c_int32, C.c_int32, C.c_int32]),
    "spc_decode_step_on_chip": (C.c_int32, [_D, C.c_int32, C.c_int32, C.c_int32]),
    "spc_decode_step": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, C.c_int32, _P, _P, _P, C.c_int32, _P, _P, _P,
                                  C.c_size_t, _P, C.c_int64, _P, C.c_int32, _P, _P]),
    "spc_decode_step_prev": (C.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, C.c_int32, _P, _P, _P, C.c_int32, _P, _P,
                                       _P, _P, C.c_size_t, _P, C.c_int64, _P, C.c_int32, _P, _P, _P, C.c_int32,
                                       _P]),
    "spc_read_device_status": (C.c_int, [_P, _D, _P]),
    "spc_rope_frequencies": (C.c_int, [C.POINTER(spc_rope_scaling), C.c_int32, _P, C.POINTER(C.c_float)]),
    "spc_rope": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spc_rope_axes": (C.c_int, [_P, C.c_int32, C.c_int32, C.c_int32, _P]),
    "spc_norm_rope": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spc_prompt_attn_workspace_bytes": (C.c_size_t, [_P]),
    "spc_prompt_attn": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "spc_prompt_attn_status": (C.c_int, [_P, _P]),
    "spc_prompt_attn_wait_limit": (C.c_int64, [C.c_int64]),
    "spc_window_attn_workspace_bytes": (C.c_size_t, [_P, C.c_int32, C.c_int32]),
    "spc_window_attn": (C.c_int, [_P, C.c_int32, C.c_int32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "spc_prefix_attn_workspace_bytes": (C.c_size_t, [_P, _P]),
    "spc_prefix_attn_together": (C.c_int32, [_P, _P, C.c_int32]),
    "spc_prefix_attn": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "spc_extend_kv": (C.c_int, [_D, C.c_int32, _P, _P, _P, _P, _P, _P, _P, C.c_int64, _P]),
    "spc_dequantize_kv": (C.c_int, [_D, _P, _P, C.c_int32, C.c_int32, _P, _P, _P, _P, _P]),
}
_CHECKED = ("spc_rope", "spc_norm_rope", "spc_prompt_attn", "spc_window_attn", "spc_prefix_attn", "spc_extend_kv",
            "spc_dequantize_kv")
_sig.update({f"{_name}_check": _sig[_name] for _name in _CHECKED})
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args
_CHECKS = {_name: getattr(_lib, f"{_name}_check") for _name in _CHECKED}


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, st):
    if st != 0:
        raise SpcError(fn, st)


def spc_abi_version() -> int:
    return int(_lib.spc_abi_version())


def spc_num_quantized(d) -> int:
    return int(_lib.spc_num_quantized(C.byref(d)))


def spc_records_bytes(d) -> int:
    return int(_lib.spc_records_bytes(C.byref(d)))


def spc_resid_bytes(d) -> int:
    return int(_lib.spc_resid_bytes(C.byref(d)))


def spc_attn_workspace_bytes(d, k_max=0) -> int:
    return int(_lib.spc_attn_workspace_bytes(C.byref(d), int(k_max)))


def spc_step_workspace_bytes(d, k_max=0) -> int:
    return int(_lib.spc_step_workspace_bytes(C.byref(d), int(k_max)))


def spc_attn_kernel_count(d, k=0, fetch_k=0) -> int:
    return int(_lib.spc_attn_kernel_count(C.byref(d), int(k), int(fetch_k)))


def spc_decode_step_kernel_count(d, k, fetch_k, next_k) -> int:
    return int(_lib.spc_decode_step_kernel_count(C.byref(d), int(k), int(fetch_k), int(next_k)))


def spc_decode_step_on_chip(d, k, fetch_k, next_k) -> int:
    """1 if spc_decode_step may be called with spec_logits=None (logits kept in TMEM)."""
    return int(_lib.spc_decode_step_on_chip(C.byref(d), int(k), int(fetch_k), int(next_k)))


def spc_decode_step(d, records, resid, q, idx, bitmap, staging, k, o, lse, spec_logits, next_k, next_idx,
                    next_bitmap, ws, ws_bytes=None, fetch_host_kv=None, fetch_n_cap=0, fetch_idx=None, fetch_k=0,
                    fetch_staging=None, stream=None, kv_self=None):
    ws_bytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("spc_decode_step",
           _lib.spc_decode_step(C.byref(d), _ptr(records), _ptr(resid), _ptr(q), _ptr(kv_self), _ptr(idx),
                                _ptr(bitmap),
                                _ptr(staging), int(k), _ptr(o), _ptr(lse), _ptr(spec_logits), int(next_k),
                                _ptr(next_idx), _ptr(next_bitmap), _ptr(ws), ws_bytes, _ptr(fetch_host_kv),
                                int(fetch_n_cap), _ptr(fetch_idx), int(fetch_k), _ptr(fetch_staging),
                                _stream(stream)))


def spc_decode_step_prev(d, records, resid, q, idx, bitmap, staging, k, o, lse, spec_logits, next_k, next_idx,
                         next_bitmap, next_src, ws, ws_bytes=None, fetch_host_kv=None, fetch_n_cap=0, fetch_idx=None,
                         fetch_k=0, fetch_staging=None, fetch_src=None, fetch_prev_staging=None, fetch_prev_k=0,
                         stream=None, kv_self=None):
    ws_bytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("spc_decode_step_prev",
           _lib.spc_decode_step_prev(C.byref(d), _ptr(records), _ptr(resid), _ptr(q), _ptr(kv_self), _ptr(idx),
                                     _ptr(bitmap), _ptr(staging), int(k), _ptr(o), _ptr(lse), _ptr(spec_logits),
                                     int(next_k), _ptr(next_idx), _ptr(next_bitmap), _ptr(next_src), _ptr(ws),
                                     ws_bytes, _ptr(fetch_host_kv), int(fetch_n_cap), _ptr(fetch_idx), int(fetch_k),
                                     _ptr(fetch_staging), _ptr(fetch_src), _ptr(fetch_prev_staging),
                                     int(fetch_prev_k), _stream(stream)))


def spc_read_device_status(ws, d, stream=None) -> int:
    """0, or SPC_ERR_TIMEOUT (6) if a bounded wait in spc_decode_step ran out (the word is cleared)."""
    return int(_lib.spc_read_device_status(_ptr(ws), C.byref(d), _stream(stream)))


def spc_quantize_kv(d, k, v, records, resid, stream=None):
    _check("spc_quantize_kv", _lib.spc_quantize_kv(C.byref(d), _ptr(k), _ptr(v), _ptr(records), _ptr(resid),
                                                   _stream(stream)))


def spc_decode_attn2(d, records, resid, q, o, lse, spec_logits, ws, ws_bytes=None, stream=None, kv_self=None):
    ws_bytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("spc_decode_attn2", _lib.spc_decode_attn2(C.byref(d), _ptr(records), _ptr(resid), _ptr(q),
                                                     _ptr(kv_self), _ptr(o), _ptr(lse), _ptr(spec_logits),
                                                     _ptr(ws), ws_bytes, _stream(stream)))


def spc_merged_attn(d, records, resid, q, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes=None,
                    stream=None, kv_self=None):
    ws_bytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("spc_merged_attn", _lib.spc_merged_attn(C.byref(d), _ptr(records), _ptr(resid), _ptr(q), _ptr(kv_self),
                                                   _ptr(idx), _ptr(bitmap), _ptr(staging), int(k), _ptr(o),
                                                   _ptr(lse), _ptr(spec_logits), _ptr(ws), ws_bytes,
                                                   _stream(stream)))


def spc_merged_attn_fetch(d, records, resid, q, idx, bitmap, staging, k, o, lse, spec_logits, ws, fetch_host_kv,
                          fetch_n_cap, fetch_idx, fetch_k, fetch_staging, ws_bytes=None, stream=None, kv_self=None):
    ws_bytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("spc_merged_attn_fetch",
           _lib.spc_merged_attn_fetch(C.byref(d), _ptr(records), _ptr(resid), _ptr(q), _ptr(kv_self), _ptr(idx),
                                      _ptr(bitmap),
                                      _ptr(staging), int(k), _ptr(o), _ptr(lse), _ptr(spec_logits), _ptr(ws),
                                      ws_bytes, _ptr(fetch_host_kv), int(fetch_n_cap), _ptr(fetch_idx),
                                      int(fetch_k), _ptr(fetch_staging), _stream(stream)))


def spc_merged_attn_fetch_prev(d, records, resid, q, idx, bitmap, staging, k, o, lse, spec_logits, ws,
                               fetch_host_kv, fetch_n_cap, fetch_idx, fetch_k, fetch_staging, fetch_src,
                               fetch_prev_staging, fetch_prev_k, ws_bytes=None, stream=None, kv_self=None):
    ws_bytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("spc_merged_attn_fetch_prev",
           _lib.spc_merged_attn_fetch_prev(C.byref(d), _ptr(records), _ptr(resid), _ptr(q), _ptr(kv_self),
                                           _ptr(idx), _ptr(bitmap), _ptr(staging), int(k), _ptr(o), _ptr(lse),
                                           _ptr(spec_logits), _ptr(ws), ws_bytes, _ptr(fetch_host_kv),
                                           int(fetch_n_cap), _ptr(fetch_idx), int(fetch_k), _ptr(fetch_staging),
                                           _ptr(fetch_src), _ptr(fetch_prev_staging), int(fetch_prev_k),
                                           _stream(stream)))


def spc_merged_attn_noalloc(d, records, resid, q, idx, bitmap, staging, k, o, lse, spec_logits, stream=None):
    """spc_merged_attn with the library's built-in workspace (for callers that cannot allocate)."""
    _check("spc_merged_attn_noalloc",
           _lib.spc_merged_attn_noalloc(C.byref(d), _ptr(records), _ptr(resid), _ptr(q), _ptr(idx), _ptr(bitmap),
                                        _ptr(staging), int(k), _ptr(o), _ptr(lse), _ptr(spec_logits),
                                        _stream(stream)))


def spc_topk_select(d, spec_logits, lse, k, idx, bitmap, stream=None):
    _check("spc_topk_select", _lib.spc_topk_select(C.byref(d), _ptr(spec_logits), _ptr(lse), int(k), _ptr(idx),
                                                   _ptr(bitmap), _stream(stream)))


def spc_topk_select_prev(d, spec_logits, lse, k, idx, bitmap, prev_idx, prev_k, src, stream=None):
    _check("spc_topk_select_prev",
           _lib.spc_topk_select_prev(C.byref(d), _ptr(spec_logits), _ptr(lse), int(k), _ptr(idx), _ptr(bitmap),
                                     _ptr(prev_idx), int(prev_k), _ptr(src), _stream(stream)))


def spc_append_kv(d, k_new, v_new, records, resid, host_kv=None, n_cap=0, stream=None):
    _check("spc_append_kv", _lib.spc_append_kv(C.byref(d), _ptr(k_new), _ptr(v_new), _ptr(records), _ptr(resid),
                                               _ptr(host_kv), int(n_cap), _stream(stream)))


def spc_offload_kv(d, k, v, host_kv, n_cap, stream=None):
    _check("spc_offload_kv", _lib.spc_offload_kv(C.byref(d), _ptr(k), _ptr(v), _ptr(host_kv), int(n_cap),
                                                 _stream(stream)))


def spc_host_gather(d, host_kv, n_cap, idx, k, staging, max_ctas=0, stream=None):
    _check("spc_host_gather", _lib.spc_host_gather(C.byref(d), _ptr(host_kv), int(n_cap), _ptr(idx), int(k),
                                                   _ptr(staging), int(max_ctas), _stream(stream)))


def spc_host_gather_prev(d, host_kv, n_cap, idx, k, staging, src, prev_staging, prev_k, max_ctas=0, stream=None):
    _check("spc_host_gather_prev",
           _lib.spc_host_gather_prev(C.byref(d), _ptr(host_kv), int(n_cap), _ptr(idx), int(k), _ptr(staging),
                                     _ptr(src), _ptr(prev_staging), int(prev_k), int(max_ctas), _stream(stream)))


# ------------------------------------------------------------------ the prompt path
# These calls take tensors of any strides (views of a fused projection, of a
# cache buffer), so they read shapes and strides from the tensors and check
# what a pointer cannot say: rank, shapes, 16-bit elements, the last axis
# contiguous, and that every tensor is on the current CUDA device.  The dims
# structs are packed in one go: short calls are bound by this marshalling.
# With _later, a list, a call is marshalled and added to it instead of made, so
# that a sequence of calls is checked in whole before its first one (_all_or_none).

ROPE_KINDS = {"plain": 0, "linear": 1, "bands": 2, "ramp": 3}
AXIS_ORDERS = {"sections": 0, "turns": 1}

_ROWS = frozenset((torch.bfloat16, torch.int16, torch.uint16))  # bf16 values or their bit patterns
_ROPE = struct.Struct("=7if18q")
_NORM_ROPE = struct.Struct("=7if18qif64s")
_PROMPT = struct.Struct("=8if4x12q")
_LAYOUT = struct.Struct("=3q")
_PREFIX = struct.Struct("=i4x6q")
assert _ROPE.size == C.sizeof(spc_rope_dims) and _NORM_ROPE.size == C.sizeof(spc_norm_rope_dims)
assert _PROMPT.size == C.sizeof(spc_prompt_dims) and _PREFIX.size == C.sizeof(spc_prefix)


def _device(fn, t):
    """The current device's index; the call's first tensor is on it."""
    if t.get_device() < 0:
        raise ValueError(f"{fn}: tensors must be on the current CUDA device, got one on {t.device}")
    return torch._C._cuda_getDevice()


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _view(fn, name, t, dev):
    """Sizes [batch, token, head, D] and strides [b, t, h] of a tensor, packed ones with a batch of 1 (an axis of one
    element has stride 0)."""
    n, st = t.shape, t.stride()
    if t.dtype not in _ROWS or t.get_device() != dev:
        raise ValueError(f"{fn}: {name} must hold bf16 rows (bfloat16, or int16 patterns) on the current CUDA device, "
                         f"got {t.dtype} on {t.device}")
    if len(n) == 4:
        (b, T, h, D), (sb, sT, sh, sd) = n, st
    elif len(n) == 3:
        (T, h, D), (sT, sh, sd) = n, st
        b, sb = 1, 0
    else:
        raise ValueError(f"{fn}: {name} must be [batch][token][head][D] (or packed, without the batch)")
    if sd != 1 and D > 1:
        raise ValueError(f"{fn}: the last axis of {name} must be contiguous")
    return b, T, h, D, (sb if b > 1 else 0, sT if T > 1 else 0, sh if h > 1 else 0)


def _like(fn, name, t, dev, ref):
    if t.shape != ref.shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(ref.shape)}")
    return _view(fn, name, t, dev)[4]


def _words(fn, name, t, dtype, n, dev):
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous {dtype} tensor of {n} elements on the current CUDA device")
    return t.data_ptr()


def spc_rope_frequencies(rot=128, theta=10000.0, kind="plain", factor=1.0, low=1.0, high=4.0, context=8192.0):
    """(turns, mscale) of a rotary rule: turns is an int64 CPU tensor (the bits
    of rot/2 64-bit fractions of a turn per position; move it to the device
    once), mscale the factor of the result.  kind: "plain", "linear",
    "bands" or "ramp" (see spc_rope_kind in include/spc.h)."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"spc_rope_frequencies: kind is one of {', '.join(ROPE_KINDS)}, got {kind!r}")
    s = spc_rope_scaling(ROPE_KINDS[kind], theta, factor, low, high, context)
    mscale = C.c_float()
    buf = (C.c_uint64 * 64)()
    _check("spc_rope_frequencies", _lib.spc_rope_frequencies(C.byref(s), int(rot), buf, C.byref(mscale)))
    return torch.tensor(buf[:int(rot) // 2], dtype=torch.int64), mscale.value  # below 2^62: positive as int64 too


def _rope_rows(fn, q, k, v, q_out, k_out, v_out):
    """(device, sizes and layouts, pointers) of the rows that a rotation reads and writes."""
    x = k if q is None else q
    if x is None:
        raise ValueError(f"{fn}: neither q nor k")
    dev = _device(fn, x)
    none = (0, 0, 0)
    ql = kl = vl = qo = ko = vo = none
    qp = kp = vp = qop = kop = vop = None
    Hq = Hkv = 0
    if q is not None:
        B, T, Hq, D, ql = _view(fn, "q", q, dev)
        qp = qop = q.data_ptr()
        qo = ql
        if q_out is not None:
            qo, qop = _like(fn, "q_out", q_out, dev, q), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError(f"{fn}: q_out without q")
    if k is not None:
        Bk, Tk, Hkv, Dk, kl = _view(fn, "k", k, dev)
        if q is None:
            B, T, D = Bk, Tk, Dk
        elif (Bk, Tk, Dk) != (B, T, D):
            raise ValueError(f"{fn}: q and k differ in batch, tokens or row")
        kp = kop = k.data_ptr()
        ko = kl
        if k_out is not None:
            ko, kop = _like(fn, "k_out", k_out, dev, k), k_out.data_ptr()
    elif k_out is not None or v is not None:
        raise ValueError(f"{fn}: k_out or v without k")
    if (v is None) != (v_out is None):
        raise ValueError(f"{fn}: v is copied, so v and v_out go together")
    if v is not None:
        vl, vo = _like(fn, "v", v, dev, k), _like(fn, "v_out", v_out, dev, k)
        vp, vop = v.data_ptr(), v_out.data_ptr()
    return dev, (B, T, Hq, Hkv, D), (*ql, *kl, *vl, *qo, *ko, *vo), (qp, kp, vp, qop, kop, vop)


def spc_rope(q, k, pos, turns, rot=128, interleaved=False, mscale=1.0, v=None, q_out=None, k_out=None, v_out=None,
             stream=None, _later=None):
    """q [B][T][Hq][D], k (and v) [B][T][Hkv][D], q or k None; the outputs of q
    and k default to in place (v is copied, so it needs v_out)."""
    fn = "spc_rope"
    dev, (B, T, Hq, Hkv, D), layouts, rows = _rope_rows(fn, q, k, v, q_out, k_out, v_out)
    pos = _words(fn, "pos", pos, torch.int32, B * T, dev)
    turns = _words(fn, "turns", turns, torch.int64, rot // 2, dev)
    if T == 0:
        return
    d = _ROPE.pack(B, T, Hq, Hkv, D, rot, 1 if interleaved else 0, mscale, *layouts)
    args = (d, pos, turns, *rows, _raw_stream(stream, dev))
    if _later is not None:
        _later.append((fn, args, None))
        return
    st = _lib.spc_rope(*args)
    if st:
        raise SpcError(fn, st)


def spc_rope_axes(sections, rot=128, order="sections"):
    """The axis of positions that turns each of the rot/2 pairs (a list, for spc_norm_rope): sections[a] pairs axis a,
    "sections" behind one another or by "turns" (see spc_axis_order in include/spc.h)."""
    if order not in AXIS_ORDERS:
        raise ValueError(f"spc_rope_axes: order is one of {', '.join(AXIS_ORDERS)}, got {order!r}")
    buf = (C.c_uint8 * 64)()
    sizes = (C.c_int32 * max(len(sections), 1))(*sections)
    _check("spc_rope_axes", _lib.spc_rope_axes(sizes, len(sections), AXIS_ORDERS[order], int(rot), buf))
    return list(buf[:int(rot) // 2])


def _axis_table(fn, axis, rot, axes):
    """The bytes of a table of axes: a sequence of any whole numbers is taken entry by entry (bytes() of an array would be
    its memory, several bytes an entry)."""
    if axis is None:
        if axes != 1:
            raise ValueError(f"{fn}: positions of {axes} axes need axis")
        return b""
    axis = list(axis)
    if len(axis) != rot // 2:
        raise ValueError(f"{fn}: axis must be {rot // 2} numbers from 0 to {axes - 1}")
    return bytes(axis)


def spc_norm_rope(q, k, pos, turns, q_weight=None, k_weight=None, eps=1e-6, axis=None, rot=128, interleaved=False,
                  mscale=1.0, v=None, q_out=None, k_out=None, v_out=None, stream=None, _later=None):
    """spc_rope with a norm of each query and key row before it.  q_weight, k_weight: fp32 [D] on the device, or None
    (rows not normed).  pos: int32 [B][T], or [axes][B][T] with axis, the axis that turns each of the rot/2 pairs (a
    sequence of rot/2 numbers; see spc_rope_axes)."""
    fn = "spc_norm_rope"
    dev, (B, T, Hq, Hkv, D), layouts, rows = _rope_rows(fn, q, k, v, q_out, k_out, v_out)
    axes = pos.shape[0] if pos.dim() == 3 else 1
    if pos.dim() == 3 and pos.shape[1:] != (B, T):  # [B][T][axes], with as many axes as sequences, has as many elements
        raise ValueError(f"{fn}: pos has shape {tuple(pos.shape)}, expected [axes][{B}][{T}]")
    axis = _axis_table(fn, axis, rot, axes)
    pos = _words(fn, "pos", pos, torch.int32, axes * B * T, dev)
    turns = _words(fn, "turns", turns, torch.int64, rot // 2, dev)
    wq, wk = _words(fn, "q_weight", q_weight, torch.float32, D, dev), _words(fn, "k_weight", k_weight, torch.float32, D, dev)
    if T == 0:
        return
    d = _NORM_ROPE.pack(B, T, Hq, Hkv, D, rot, 1 if interleaved else 0, mscale, *layouts, axes, eps, axis)
    args = (d, pos, turns, wq, wk, *rows, _raw_stream(stream, dev))
    if _later is not None:
        _later.append((fn, args, None))
        return
    st = _lib.spc_norm_rope(*args)
    if st:
        raise SpcError(fn, st)


def _prompt_dims(fn, q, k, v, o, S, q_max, k_max, scale, dev):
    qs, qt, Hq, D, ql = _view(fn, "q", q, dev)
    ks, kt, Hkv, Dk, kl = _view(fn, "k", k, dev)
    vl, ol = _like(fn, "v", v, dev, k), _like(fn, "o", o, dev, q)
    if Dk != D or D == 0:
        raise ValueError(f"{fn}: q has rows of {D} elements, k of {Dk}")
    if (qs != S and q.dim() == 4) or (ks != S and k.dim() == 4):
        raise ValueError(f"{fn}: batches of {qs} and {ks}, and there are {S} sequences")
    return _PROMPT.pack(S, Hq, Hkv, D, qt, kt, qt if q_max is None else q_max, kt if k_max is None else k_max,
                        D ** -0.5 if scale is None else scale, *ql, *kl, *vl, *ol)


def _sequences(q, k, *words):
    for t in words:
        if t is not None:
            return t.numel()
    return q.shape[0] if q.dim() == 4 else k.shape[0] if k.dim() == 4 else 1


def spc_prompt_attn_workspace_bytes(q, k, v, o, S=None, q_max=None, k_max=None) -> int:
    """Bytes of workspace of spc_prompt_attn over these tensors (S sequences; default: the batch)."""
    fn = "spc_prompt_attn_workspace_bytes"
    d = _prompt_dims(fn, q, k, v, o, _sequences(q, k) if S is None else S, q_max, k_max, None, _device(fn, q))
    return int(_lib.spc_prompt_attn_workspace_bytes(d))


def _attend(fn, call, size, rule, prefix, q, k, v, o, lse, q_begin, q_len, k_begin, k_len, q_max, k_max, scale, ws, ws_bytes, stream,
            later):
    """A call of spc_prompt_attn or one of its siblings: call and size, the library's functions; rule, its arguments behind
    the dims, and prefix, those between the queries and the keys."""
    dev = _device(fn, q)
    S = _sequences(q, k, q_len, k_len, q_begin, k_begin)
    d = _prompt_dims(fn, q, k, v, o, S, q_max, k_max, scale, dev)
    i32 = torch.int32
    qb, ql = _words(fn, "q_begin", q_begin, i32, S, dev), _words(fn, "q_len", q_len, i32, S, dev)
    kb, kl = _words(fn, "k_begin", k_begin, i32, S, dev), _words(fn, "k_len", k_len, i32, S, dev)
    lse_ptr = None if lse is None else _words(fn, "lse", lse, torch.float32, q.numel() // max(q.shape[-1], 1), dev)
    s = _raw_stream(stream, dev)
    own = None
    if ws is None:
        if stream is not None and s != _raw_stream(None, dev):
            raise ValueError(f"{fn}: a call on another stream than the current one needs ws")
        w, ws_bytes = None, size(d, *rule)
        if ws_bytes > 256:  # the keys are split; else the call needs none
            w = own = torch._C._cuda_cudaCachingAllocator_raw_alloc(ws_bytes, s)  # a tensor's allocation takes 3 us more
        else:
            ws_bytes = 0
    else:
        w = _ptr(ws)
        if not isinstance(ws, int):
            if ws.get_device() != dev or not ws.is_contiguous():
                raise ValueError(f"{fn}: ws must be contiguous on the current CUDA device")
            if ws_bytes is None:
                ws_bytes = ws.numel() * ws.element_size()
        elif ws_bytes is None:
            raise ValueError(f"{fn}: a workspace given by its address needs ws_bytes")
    args = (d, *rule, q.data_ptr(), *prefix, k.data_ptr(), v.data_ptr(), qb, ql, kb, kl, o.data_ptr(), lse_ptr, w, ws_bytes, s)
    if later is not None:
        later.append((fn, args, own))
        return
    try:
        st = call(*args)
    finally:
        if own is not None:
            torch._C._cuda_cudaCachingAllocator_raw_delete(own)
    if st:
        raise SpcError(fn, st)


def spc_prompt_attn(q, k, v, o, lse=None, q_begin=None, q_len=None, k_begin=None, k_len=None, q_max=None, k_max=None,
                    scale=None, ws=None, ws_bytes=None, stream=None, _later=None):
    """q and o: [T][Hq][D] (packed sequences) or [S][T][Hq][D]; k and v
    [T][Hkv][D] or [S][T][Hkv][D].  q_begin, q_len, k_begin, k_len: int32 [S]
    on the device, or None.  q_max, k_max bound the lengths (default: the
    token axis).  lse: fp32 of o's shape without D, contiguous.  Without ws a
    workspace, where one is needed, is taken from torch's allocator for the
    call, which needs the call to be on the current stream; a wait that ran
    out is then found by spc_prompt_attn_status() of the device."""
    _attend("spc_prompt_attn", _lib.spc_prompt_attn, _lib.spc_prompt_attn_workspace_bytes, (), (), q, k, v, o, lse, q_begin,
            q_len, k_begin, k_len, q_max, k_max, scale, ws, ws_bytes, stream, _later)


def _window(fn, window, sinks):
    if not 1 <= window or sinks < 0:
        raise ValueError(f"{fn}: a window of at least 1 and no negative number of first tokens, got {window} and {sinks}")
    return min(window, 2 ** 31 - 1), min(sinks, 2 ** 31 - 1)


def spc_window_attn_workspace_bytes(q, k, v, o, window, sinks=0, S=None, q_max=None, k_max=None) -> int:
    """Bytes of workspace of spc_window_attn over these tensors (S sequences; default: the batch)."""
    fn = "spc_window_attn_workspace_bytes"
    d = _prompt_dims(fn, q, k, v, o, _sequences(q, k) if S is None else S, q_max, k_max, None, _device(fn, q))
    return int(_lib.spc_window_attn_workspace_bytes(d, *_window(fn, window, sinks)))


def spc_window_attn(q, k, v, o, window, sinks=0, lse=None, q_begin=None, q_len=None, k_begin=None, k_len=None, q_max=None,
                    k_max=None, scale=None, ws=None, ws_bytes=None, stream=None, _later=None):
    """spc_prompt_attn where a query sees the last `window` keys up to its own
    and the first `sinks` keys of its sequence; the other arguments are
    spc_prompt_attn's."""
    fn = "spc_window_attn"
    _attend(fn, _lib.spc_window_attn, _lib.spc_window_attn_workspace_bytes, _window(fn, window, sinks), (), q, k, v, o, lse,
            q_begin, q_len, k_begin, k_len, q_max, k_max, scale, ws, ws_bytes, stream, _later)


def _prefix(fn, pk, pv, k, dev):
    """The packed spc_prefix of a call's shared rows."""
    _, P, Hkv, D, lk = _view(fn, "pk", pk, dev)
    if pk.dim() != 3 or (Hkv, D) != (k.shape[-2], k.shape[-1]):
        raise ValueError(f"{fn}: pk has shape {tuple(pk.shape)}, expected [P][{k.shape[-2]}][{k.shape[-1]}]")
    return _PREFIX.pack(P, *lk, *_like(fn, "pv", pv, dev, pk))


def spc_prefix_attn_workspace_bytes(q, pk, pv, k, v, o, S=None, q_max=None, k_max=None) -> int:
    """Bytes of workspace of spc_prefix_attn over these tensors (S sequences; default: the batch)."""
    fn = "spc_prefix_attn_workspace_bytes"
    dev = _device(fn, q)
    d = _prompt_dims(fn, q, k, v, o, _sequences(q, k) if S is None else S, q_max, k_max, None, dev)
    return int(_lib.spc_prefix_attn_workspace_bytes(d, _prefix(fn, pk, pv, k, dev)))


def spc_prefix_attn_together(q, pk, pv, k, v, o, S=None, q_max=None, k_max=None, placed=False) -> int:
    """Whether spc_prefix_attn over these tensors (placed: with a q_begin) walks over the prefix once for all sequences' rows
    (2: with their own keys in the same walk, 1: these in a launch of their own) or for each sequence (0)."""
    fn = "spc_prefix_attn_together"
    dev = _device(fn, q)
    d = _prompt_dims(fn, q, k, v, o, _sequences(q, k) if S is None else S, q_max, k_max, None, dev)
    return int(_lib.spc_prefix_attn_together(d, _prefix(fn, pk, pv, k, dev), 1 if placed else 0))


def spc_prefix_attn(q, pk, pv, k, v, o, lse=None, p_len=None, q_begin=None, q_len=None, k_begin=None, k_len=None,
                    q_max=None, k_max=None, scale=None, ws=None, ws_bytes=None, stream=None, _later=None):
    """spc_prompt_attn of sequences that share a prefix: pk, pv [P][Hkv][D],
    which every query sees in whole; k and v are the sequences' own keys behind
    it.  p_len: int32 [1] on the device (how many of the P tokens there are), or
    None.  The other arguments are spc_prompt_attn's."""
    fn = "spc_prefix_attn"
    dev = _device(fn, q)
    p = _prefix(fn, pk, pv, k, dev)
    n = _words(fn, "p_len", p_len, torch.int32, 1, dev)
    _attend(fn, _lib.spc_prefix_attn, _lib.spc_prefix_attn_workspace_bytes, (p,), (pk.data_ptr(), pv.data_ptr(), n), q, k, v, o,
            lse, q_begin, q_len, k_begin, k_len, q_max, k_max, scale, ws, ws_bytes, stream, _later)


def spc_prompt_attn_status(ws=None, stream=None) -> int:
    """0, or SPC_ERR_TIMEOUT (6) if a bounded wait in spc_prompt_attn ran out (the word is cleared): in a call with this
    workspace, or, without one, in any call on the current device."""
    return int(_lib.spc_prompt_attn_status(_ptr(ws), _stream(stream)))


def spc_prompt_attn_wait_limit(ns=0) -> int:
    """The limit in ns of a wait in spc_prompt_attn's kernels before this call; ns > 0 sets it for the calls to come."""
    return int(_lib.spc_prompt_attn_wait_limit(int(ns)))


def _cache_call(fn, d, names, k, v, records, resid):
    """(n, packed layouts of k and v, pointers of the cache, device) of a call on a run of tokens."""
    dev = _device(fn, k)
    B, n, h, D, kl = _view(fn, names[0], k, dev)
    if k.dim() != 4 or (B, h, D) != (d.B, d.Hkv, d.D):
        raise ValueError(f"{fn}: {names[0]} has shape {tuple(k.shape)}, expected [{d.B}][n][{d.Hkv}][{d.D}]")
    vl = _like(fn, names[1], v, dev, k)
    ptr = []
    for name, t, need in (("records", records, _lib.spc_records_bytes), ("resid", resid, _lib.spc_resid_bytes)):
        if t is None or isinstance(t, int):
            ptr.append(t)
            continue
        if t.get_device() != dev or not t.is_contiguous() or t.numel() * t.element_size() < need(C.byref(d)):
            raise ValueError(f"{fn}: {name} must be contiguous on the current CUDA device and hold {need(C.byref(d))} bytes")
        ptr.append(t.data_ptr())
    return n, _LAYOUT.pack(*kl), _LAYOUT.pack(*vl), ptr, dev


def spc_extend_kv(d, k_new, v_new, records, resid, host_kv=None, n_cap=0, stream=None, _later=None):
    """k_new, v_new: 16-bit [B][n][Hkv][D] of any strides; the caller advances d.N by n."""
    fn = "spc_extend_kv"
    n, lk, lv, (rec, res), dev = _cache_call(fn, d, ("k_new", "v_new"), k_new, v_new, records, resid)
    args = (C.byref(d), n, k_new.data_ptr(), v_new.data_ptr(), lk, lv, rec, res, _ptr(host_kv), n_cap,
            _raw_stream(stream, dev))
    if _later is not None:
        _later.append((fn, args, None))
        return
    st = _lib.spc_extend_kv(*args)
    if st:
        raise SpcError(fn, st)


def spc_dequantize_kv(d, records, resid, first, k, v, stream=None, _later=None):
    """k, v: 16-bit [B][n][Hkv][D] of any strides, for the tokens first .. first+n-1."""
    fn = "spc_dequantize_kv"
    n, lk, lv, (rec, res), dev = _cache_call(fn, d, ("k", "v"), k, v, records, resid)
    args = (C.byref(d), rec, res, first, n, k.data_ptr(), v.data_ptr(), lk, lv, _raw_stream(stream, dev))
    if _later is not None:
        _later.append((fn, args, None))
        return
    st = _lib.spc_dequantize_kv(*args)
    if st:
        raise SpcError(fn, st)


@contextlib.contextmanager
def _all_or_none():
    """A list for calls' _later: they are made in order at the end of the block, unless one of them is refused, there or
    by its check; then none is.  Workspaces that they took are freed in any case."""
    calls = []
    try:
        yield calls
        for fn, args, _ in calls:
            _check(fn, _CHECKS[fn](*args))
        for fn, args, _ in calls:
            _check(fn, getattr(_lib, fn)(*args))
    finally:
        for _, _, own in calls:
            if own is not None:
                torch._C._cuda_cudaCachingAllocator_raw_delete(own)
