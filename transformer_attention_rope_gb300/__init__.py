"""GB300-native APEX-1 attention block: RoPE + GQA + causal/sliding-window SDPA.

This package is a thin ctypes binding over the C ABI declared in
``include/apex_attn.h`` (``_build/libapex_attn.so``).  It only marshals
arguments: every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback -- if the library is missing, every call raises.

Raw C-ABI names (pointers and sizes):
    apex_attn_fwd, apex_attn_decode, apex_attn_decode_noalloc, apex_attn_decode_workspace_bytes,
    apex_attn_rope_reserve, apex_attn_device_status, apex_attn_status_string,
    apex_attn_fwd_ex, apex_attn_fwd_ws, apex_attn_fwd_workspace_bytes, apex_attn_decode_ex, apex_attn_rope_keys,
    apex_attn_mla_fwd, apex_attn_mla_fwd_ws, apex_attn_mla_fwd_workspace_bytes, apex_attn_mla_decode,
    apex_attn_mla_rope_keys (with an Options struct),
    apex_attn_sink_fwd, apex_attn_sink_fwd_workspace_bytes, apex_attn_sink_decode, apex_attn_sink_tree_decode (windows
    with sinks),
    apex_attn_rope (with RopeOptions and RopeTensor structs), apex_attn_tree_decode, apex_attn_tree_workspace_bytes,
    apex_attn_decode_weights, apex_attn_decode_weights_workspace_bytes, apex_attn_evict,
    apex_attn_evict_workspace_bytes, apex_attn_norm_rope and apex_attn_norm_rope_grad (with NormTensor structs),
    apex_attn_norm_rope_grad_workspace_bytes, apex_attn_append4 and apex_attn_unpack4 (with Bits4Tensor structs),
    apex_attn_decode4, apex_attn_decode4_workspace_bytes
Tensor conveniences (torch, bf16, contiguous, on their own CUDA device):
    fwd(q, k, v, ...), decode(q, k_cache, v_cache, q_pos, ...), rope_keys(k, ...), mla_fwd(q, k, v, d_r, ...),
    mla_decode(q, k_cache, v_cache, q_pos, d_r, ...), mla_rope_keys(k, d_r, ...)
Over caches of rotated keys (int32 lengths and positions on the device; the tensors' own device):
    rope(q, k, v, positions=...), norm_rope(q, k, v, positions=..., q_weight=..., k_weight=...) and its gradient
    norm_rope_grad(q_grad, q, k_grad, k, positions=...), tree_decode(q, k_cache, v_cache, lens, ...),
    decode_weights(q, k_cache, v_cache, lens, acc, ...), evict(k_cache, v_cache, acc, lens, budget, ...)
Over caches held in 4 bits:
    append4(k, v, k4, k_scale, v4, v_scale, row0=...), unpack4(k4, k_scale, v4, v_scale, row0=..., n_rows=...),
    decode4(q, k4, k_scale, v4, v_scale, lens, ...)
No call is recorded by autograd: results do not require gradients, whatever their inputs do.  The gradient of
rope is rope with inverse=True, that of norm_rope is norm_rope_grad.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

__all__ = [
    "ApexError", "library_path", "load_library", "apex_attn_fwd", "apex_attn_decode", "apex_attn_decode_noalloc",
    "apex_attn_decode_workspace_bytes", "apex_attn_rope_reserve", "apex_attn_device_status",
    "apex_attn_status_string", "apex_attn_fwd_ex", "apex_attn_fwd_ws", "apex_attn_fwd_workspace_bytes",
    "apex_attn_decode_ex", "apex_attn_rope_keys", "fwd_workspace_bytes",
    "apex_attn_mla_fwd", "apex_attn_mla_fwd_ws", "apex_attn_mla_fwd_workspace_bytes", "apex_attn_mla_decode",
    "apex_attn_mla_rope_keys", "apex_attn_selftest_wait_timeout", "Options", "fwd", "decode",
    "decode_workspace_bytes", "mla_fwd_workspace_bytes",
    "rope_keys", "mla_fwd", "mla_decode", "mla_rope_keys",
    "apex_attn_rope", "apex_attn_tree_decode", "apex_attn_tree_workspace_bytes", "apex_attn_decode_weights",
    "apex_attn_decode_weights_workspace_bytes", "apex_attn_evict", "apex_attn_evict_workspace_bytes",
    "RopeOptions", "RopeTensor", "rope", "tree_decode", "tree_workspace_bytes", "decode_weights",
    "decode_weights_workspace_bytes", "evict", "evict_workspace_bytes",
    "apex_attn_norm_rope", "apex_attn_norm_rope_grad", "apex_attn_norm_rope_grad_workspace_bytes", "NormTensor",
    "norm_rope", "norm_rope_grad", "norm_rope_grad_workspace_bytes",
    "apex_attn_append4", "apex_attn_unpack4", "apex_attn_decode4", "apex_attn_decode4_workspace_bytes", "Bits4Tensor",
    "append4", "unpack4", "decode4", "decode4_workspace_bytes",
    "apex_attn_sink_fwd", "apex_attn_sink_fwd_workspace_bytes", "apex_attn_sink_decode", "apex_attn_sink_tree_decode",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libapex_attn.so")
_lock = threading.Lock()
_lib = None
_torch = None  # the torch module, once a call over caches of rotated keys has needed it

APEX_OK = 0
_STATUS_NAMES = {0: "APEX_OK", 1: "APEX_ERR_INVALID_ARG", 2: "APEX_ERR_UNSUPPORTED", 3: "APEX_ERR_CUDA",
                 4: "APEX_ERR_NO_MEMORY", 5: "APEX_ERR_DEVICE_TIMEOUT"}


class Options(ctypes.Structure):
    """apex_attn_options of include/apex_attn.h (all zeros: the plain block)."""
    _fields_ = [("window", ctypes.c_int), ("q_pos", ctypes.c_int), ("rope_base", ctypes.c_float),
                ("yarn_scale", ctypes.c_float), ("yarn_beta_fast", ctypes.c_float),
                ("yarn_beta_slow", ctypes.c_float), ("prefix_len", ctypes.c_int), ("keys_prerotated", ctypes.c_int)]


class RopeOptions(ctypes.Structure):
    """apex_rope_options of include/apex_attn.h (all zeros: interleaved, whole rows, base 10000)."""
    _fields_ = [("layout", ctypes.c_int), ("rot_start", ctypes.c_int), ("d_rot", ctypes.c_int),
                ("inverse", ctypes.c_int), ("rope_base", ctypes.c_float), ("linear_scale", ctypes.c_float),
                ("yarn_scale", ctypes.c_float), ("yarn_beta_fast", ctypes.c_float),
                ("yarn_beta_slow", ctypes.c_float)]


class RopeTensor(ctypes.Structure):
    """apex_rope_tensor of include/apex_attn.h (strides in elements)."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n_heads", ctypes.c_int),
                ("d_row", ctypes.c_int)] + [(n, ctypes.c_longlong) for n in ("in_b", "in_h", "in_s", "out_b",
                                                                             "out_h", "out_s")]


class NormTensor(ctypes.Structure):
    """apex_norm_tensor of include/apex_attn.h (strides in elements)."""
    _fields_ = [("x", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("dweight", ctypes.c_void_p), ("n_heads", ctypes.c_int),
                ("d_row", ctypes.c_int), ("weight_f32", ctypes.c_int), ("weight_per_head", ctypes.c_int)] + \
               [(n, ctypes.c_longlong) for n in ("x_b", "x_h", "x_s", "dy_b", "dy_h", "dy_s", "out_b", "out_h",
                                                 "out_s")]


class Bits4Tensor(ctypes.Structure):
    """apex_bits4_tensor of include/apex_attn.h (strides in elements)."""
    _fields_ = [("rows", ctypes.c_void_p), ("bytes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("factor", ctypes.c_void_p), ("b", ctypes.c_longlong), ("h", ctypes.c_longlong),
                ("s", ctypes.c_longlong), ("d", ctypes.c_int)]


class ApexError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (what, _STATUS_NAMES.get(status, status),
                                                 apex_attn_status_string(status)))


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load the CUDA library; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError("libapex_attn.so is not built (run __graft_entry__.build() or "
                                   "python transformer_attention_rope_gb300/build.py); there is no fallback")
            lib = ctypes.CDLL(_LIB_PATH)
            vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            lib.apex_attn_fwd.argtypes = [vp, vp, vp, vp] + [i32] * 8 + [f32, vp]
            lib.apex_attn_fwd.restype = i32
            lib.apex_attn_decode.argtypes = [vp, vp, vp, vp] + [i32] * 7 + [f32, vp, sz, vp]
            lib.apex_attn_decode.restype = i32
            lib.apex_attn_decode_noalloc.argtypes = [vp, vp, vp, vp] + [i32] * 7 + [f32, vp]
            lib.apex_attn_decode_noalloc.restype = i32
            op = ctypes.POINTER(Options)
            lib.apex_attn_fwd_ex.argtypes = [vp, vp, vp, vp] + [i32] * 6 + [op, vp]
            lib.apex_attn_fwd_ex.restype = i32
            lib.apex_attn_fwd_ws.argtypes = [vp, vp, vp, vp] + [i32] * 6 + [op, vp, sz, vp]
            lib.apex_attn_fwd_ws.restype = i32
            lib.apex_attn_fwd_workspace_bytes.argtypes = [i32] * 6 + [op]
            lib.apex_attn_fwd_workspace_bytes.restype = sz
            lib.apex_attn_mla_fwd.argtypes = [vp, vp, vp, vp] + [i32] * 7 + [op, vp]
            lib.apex_attn_mla_fwd.restype = i32
            lib.apex_attn_mla_fwd_ws.argtypes = [vp, vp, vp, vp] + [i32] * 7 + [op, vp, sz, vp]
            lib.apex_attn_mla_fwd_ws.restype = i32
            lib.apex_attn_mla_fwd_workspace_bytes.argtypes = [i32] * 7 + [op]
            lib.apex_attn_mla_fwd_workspace_bytes.restype = sz
            lib.apex_attn_mla_decode.argtypes = [vp, vp, vp, vp] + [i32] * 6 + [op, vp, sz, vp]
            lib.apex_attn_mla_decode.restype = i32
            lib.apex_attn_sink_fwd.argtypes = [vp, vp, vp, vp] + [i32] * 8 + [op, vp, sz, vp]
            lib.apex_attn_sink_fwd.restype = i32
            lib.apex_attn_sink_fwd_workspace_bytes.argtypes = [i32] * 8 + [op]
            lib.apex_attn_sink_fwd_workspace_bytes.restype = sz
            lib.apex_attn_sink_decode.argtypes = [vp, vp, vp, vp] + [i32] * 7 + [op, vp, sz, vp]
            lib.apex_attn_sink_decode.restype = i32
            lib.apex_attn_decode_ex.argtypes = [vp, vp, vp, vp] + [i32] * 5 + [op, vp, sz, vp]
            lib.apex_attn_decode_ex.restype = i32
            lib.apex_attn_rope_keys.argtypes = [vp, vp] + [i32] * 4 + [ctypes.c_longlong] * 2 + [op, vp]
            lib.apex_attn_rope_keys.restype = i32
            lib.apex_attn_mla_rope_keys.argtypes = [vp, vp] + [i32] * 5 + [ctypes.c_longlong] * 2 + [op, vp]
            lib.apex_attn_mla_rope_keys.restype = i32
            i64 = ctypes.c_longlong
            # the structs by address: byref(...) or their bytes
            lib.apex_attn_rope.argtypes = [vp, vp, vp, i32, i32, vp, i64, vp, i32, vp, vp]
            lib.apex_attn_rope.restype = i32
            lib.apex_attn_norm_rope.argtypes = [vp, vp, vp, i32, i32, vp, i64, vp, i32, vp, f32, vp]
            lib.apex_attn_norm_rope.restype = i32
            lib.apex_attn_norm_rope_grad.argtypes = [vp, vp, i32, i32, vp, i64, vp, f32, vp, sz, vp]
            lib.apex_attn_norm_rope_grad.restype = i32
            lib.apex_attn_norm_rope_grad_workspace_bytes.argtypes = [i32] * 4
            lib.apex_attn_norm_rope_grad_workspace_bytes.restype = sz
            for move in (lib.apex_attn_append4, lib.apex_attn_unpack4):
                move.argtypes = [vp, vp] + [i32] * 4 + [vp, vp]
                move.restype = i32
            lib.apex_attn_decode4.argtypes = [vp] * 6 + [i32] * 7 + [vp, i32, i32, vp, vp, f32, vp, sz, vp]
            lib.apex_attn_decode4.restype = i32
            lib.apex_attn_decode4_workspace_bytes.argtypes = [i32] * 7
            lib.apex_attn_decode4_workspace_bytes.restype = sz
            lib.apex_attn_tree_decode.argtypes = [vp] * 4 + [i32] * 7 + [vp, vp, i64, vp, i32, f32, vp, sz, vp]
            lib.apex_attn_tree_decode.restype = i32
            lib.apex_attn_sink_tree_decode.argtypes = [vp] * 4 + [i32] * 7 + [vp, vp, i64, vp, i32, i32, f32, vp, sz, vp]
            lib.apex_attn_sink_tree_decode.restype = i32
            lib.apex_attn_tree_workspace_bytes.argtypes = [i32] * 7
            lib.apex_attn_tree_workspace_bytes.restype = sz
            lib.apex_attn_decode_weights.argtypes = [vp] * 4 + [i32] * 6 + [vp, vp, f32, vp, sz, vp]
            lib.apex_attn_decode_weights.restype = i32
            lib.apex_attn_decode_weights_workspace_bytes.argtypes = [i32] * 6
            lib.apex_attn_decode_weights_workspace_bytes.restype = sz
            lib.apex_attn_evict.argtypes = [vp, vp] + [i32] * 5 + [vp] * 4 + [i32] * 3 + [vp] * 4 + [sz, vp]
            lib.apex_attn_evict.restype = i32
            lib.apex_attn_evict_workspace_bytes.argtypes = [i32] * 4
            lib.apex_attn_evict_workspace_bytes.restype = sz
            lib.apex_attn_decode_workspace_bytes.argtypes = [i32] * 5
            lib.apex_attn_decode_workspace_bytes.restype = sz
            lib.apex_attn_rope_reserve.argtypes = [i32, i32, f32]
            lib.apex_attn_rope_reserve.restype = i32
            lib.apex_attn_selftest_wait_timeout.argtypes = [i32, vp]
            lib.apex_attn_selftest_wait_timeout.restype = i32
            lib.apex_attn_device_status.argtypes = []
            lib.apex_attn_device_status.restype = i32
            lib.apex_attn_status_string.argtypes = [i32]
            lib.apex_attn_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


# ------------------------------------------------------------------ raw C ABI
def apex_attn_fwd(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, window, q_pos0, rope_base, stream) -> int:
    return load_library().apex_attn_fwd(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, window, q_pos0,
                                        rope_base, stream)


def apex_attn_decode(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, window, q_pos, rope_base,
                     workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_decode(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, window, q_pos,
                                           rope_base, workspace, workspace_bytes, stream)


def apex_attn_decode_noalloc(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, window, q_pos, rope_base,
                             stream) -> int:
    return load_library().apex_attn_decode_noalloc(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, window,
                                                   q_pos, rope_base, stream)


def apex_attn_fwd_ex(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, opt, stream) -> int:
    return load_library().apex_attn_fwd_ex(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h,
                                           ctypes.byref(opt) if opt is not None else None, stream)


def apex_attn_fwd_ws(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, opt, workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_fwd_ws(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h,
                                           ctypes.byref(opt) if opt is not None else None, workspace,
                                           workspace_bytes, stream)


def apex_attn_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, opt) -> int:
    return load_library().apex_attn_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h,
                                                        ctypes.byref(opt) if opt is not None else None)


def apex_attn_mla_fwd(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, d_r, opt, stream) -> int:
    return load_library().apex_attn_mla_fwd(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, d_r,
                                            ctypes.byref(opt) if opt is not None else None, stream)


def apex_attn_mla_fwd_ws(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, d_r, opt, workspace, workspace_bytes,
                         stream) -> int:
    return load_library().apex_attn_mla_fwd_ws(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, d_r,
                                               ctypes.byref(opt) if opt is not None else None, workspace,
                                               workspace_bytes, stream)


def apex_attn_mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, d_r, opt) -> int:
    return load_library().apex_attn_mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, d_r,
                                                            ctypes.byref(opt) if opt is not None else None)


def apex_attn_mla_decode(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, d_r, opt, workspace,
                         workspace_bytes, stream) -> int:
    return load_library().apex_attn_mla_decode(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, d_r,
                                               ctypes.byref(opt) if opt is not None else None, workspace,
                                               workspace_bytes, stream)


def apex_attn_sink_fwd(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, d_r, n_sink, opt, workspace, workspace_bytes,
                       stream) -> int:
    return load_library().apex_attn_sink_fwd(q, k, v, out, B, H_q, H_kv, S_q, S_k, d_h, d_r, n_sink,
                                             ctypes.byref(opt) if opt is not None else None, workspace,
                                             workspace_bytes, stream)


def apex_attn_sink_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, d_r, n_sink, opt) -> int:
    return load_library().apex_attn_sink_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, d_r, n_sink,
                                                             ctypes.byref(opt) if opt is not None else None)


def apex_attn_sink_decode(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, d_r, n_sink, opt, workspace,
                          workspace_bytes, stream) -> int:
    return load_library().apex_attn_sink_decode(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, d_r, n_sink,
                                                ctypes.byref(opt) if opt is not None else None, workspace,
                                                workspace_bytes, stream)


def apex_attn_decode_ex(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h, opt, workspace, workspace_bytes,
                        stream) -> int:
    return load_library().apex_attn_decode_ex(q, k_cache, v_cache, out, B, H_q, H_kv, S_k, d_h,
                                              ctypes.byref(opt) if opt is not None else None, workspace,
                                              workspace_bytes, stream)


def apex_attn_rope_keys(k_in, k_out, n_heads, n_pos, d_h, pos0, in_head_stride, out_head_stride, opt,
                        stream) -> int:
    return load_library().apex_attn_rope_keys(k_in, k_out, n_heads, n_pos, d_h, pos0, in_head_stride,
                                              out_head_stride, ctypes.byref(opt) if opt is not None else None,
                                              stream)


def apex_attn_mla_rope_keys(k_in, k_out, n_heads, n_pos, d_h, d_r, pos0, in_head_stride, out_head_stride, opt,
                            stream) -> int:
    return load_library().apex_attn_mla_rope_keys(k_in, k_out, n_heads, n_pos, d_h, d_r, pos0, in_head_stride,
                                                  out_head_stride, ctypes.byref(opt) if opt is not None else None,
                                                  stream)


def apex_attn_rope(q, k, v, B, S, positions, pos_stride, row0, out_rows, opt, stream) -> int:
    ref = [ctypes.byref(t) if isinstance(t, ctypes.Structure) else t for t in (q, k, v, opt)]
    return load_library().apex_attn_rope(ref[0], ref[1], ref[2], B, S, positions, pos_stride, row0, out_rows, ref[3],
                                         stream)


def apex_attn_norm_rope(q, k, v, B, S, positions, pos_stride, row0, out_rows, opt, eps, stream) -> int:
    ref = [ctypes.byref(t) if isinstance(t, ctypes.Structure) else t for t in (q, k, v, opt)]
    return load_library().apex_attn_norm_rope(ref[0], ref[1], ref[2], B, S, positions, pos_stride, row0, out_rows,
                                              ref[3], eps, stream)


def apex_attn_norm_rope_grad(q, k, B, S, positions, pos_stride, opt, eps, workspace, workspace_bytes, stream) -> int:
    ref = [ctypes.byref(t) if isinstance(t, ctypes.Structure) else t for t in (q, k, opt)]
    return load_library().apex_attn_norm_rope_grad(ref[0], ref[1], B, S, positions, pos_stride, ref[2], eps, workspace,
                                                   workspace_bytes, stream)


def apex_attn_norm_rope_grad_workspace_bytes(H_q, H_kv, d_q, d_k) -> int:
    return load_library().apex_attn_norm_rope_grad_workspace_bytes(H_q, H_kv, d_q, d_k)


def apex_attn_append4(k, v, B, H_kv, S, S_cap, row0, stream) -> int:
    ref = [ctypes.byref(t) if isinstance(t, ctypes.Structure) else t for t in (k, v)]
    return load_library().apex_attn_append4(ref[0], ref[1], B, H_kv, S, S_cap, row0, stream)


def apex_attn_unpack4(k, v, B, H_kv, S, S_cap, row0, stream) -> int:
    ref = [ctypes.byref(t) if isinstance(t, ctypes.Structure) else t for t in (k, v)]
    return load_library().apex_attn_unpack4(ref[0], ref[1], B, H_kv, S, S_cap, row0, stream)


def apex_attn_decode4(q, k4, k_scale, v4, v_scale, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens, window, n_sink,
                      k_factor, v_factor, scale, workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_decode4(q, k4, k_scale, v4, v_scale, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens,
                                            window, n_sink, k_factor, v_factor, scale, workspace, workspace_bytes,
                                            stream)


def apex_attn_decode4_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v) -> int:
    return load_library().apex_attn_decode4_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v)


def apex_attn_tree_decode(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens, tree_mask, mask_stride,
                          positions, window, scale, workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_tree_decode(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens,
                                                tree_mask, mask_stride, positions, window, scale, workspace,
                                                workspace_bytes, stream)


def apex_attn_sink_tree_decode(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens, tree_mask,
                               mask_stride, positions, window, n_sink, scale, workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_sink_tree_decode(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens,
                                                     tree_mask, mask_stride, positions, window, n_sink, scale,
                                                     workspace, workspace_bytes, stream)


def apex_attn_tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v) -> int:
    return load_library().apex_attn_tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v)


def apex_attn_decode_weights(q, k_cache, v_cache, out, B, H_q, H_kv, S_cap, d_qk, d_v, lens, acc, scale, workspace,
                             workspace_bytes, stream) -> int:
    return load_library().apex_attn_decode_weights(q, k_cache, v_cache, out, B, H_q, H_kv, S_cap, d_qk, d_v, lens,
                                                   acc, scale, workspace, workspace_bytes, stream)


def apex_attn_decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_v) -> int:
    return load_library().apex_attn_decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_v)


def apex_attn_evict(k_cache, v_cache, B, H_kv, S_cap, d_k, d_v, acc, positions, lens, next_pos, budget, n_sink,
                    n_recent, acc_out, positions_out, lens_out, workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_evict(k_cache, v_cache, B, H_kv, S_cap, d_k, d_v, acc, positions, lens, next_pos,
                                          budget, n_sink, n_recent, acc_out, positions_out, lens_out, workspace,
                                          workspace_bytes, stream)


def apex_attn_evict_workspace_bytes(B, H_kv, S_cap, budget) -> int:
    return load_library().apex_attn_evict_workspace_bytes(B, H_kv, S_cap, budget)


def apex_attn_decode_workspace_bytes(B, H_q, H_kv, S_k, d_h) -> int:
    return load_library().apex_attn_decode_workspace_bytes(B, H_q, H_kv, S_k, d_h)


def apex_attn_rope_reserve(max_pos, d_h, rope_base) -> int:
    return load_library().apex_attn_rope_reserve(max_pos, d_h, rope_base)


def apex_attn_selftest_wait_timeout(timeout_ms, stream) -> int:
    return load_library().apex_attn_selftest_wait_timeout(timeout_ms, stream)


def apex_attn_device_status() -> int:
    return load_library().apex_attn_device_status()


def apex_attn_status_string(status: int) -> str:
    return load_library().apex_attn_status_string(int(status)).decode()


# ------------------------------------------------------------------ torch conveniences
def _options(window=0, q_pos=0, rope_base=10000.0, yarn_scale=1.0, yarn_beta_fast=32.0, yarn_beta_slow=1.0,
             prefix_len=0, keys_prerotated=False) -> Options:
    return Options(_window(window), _int32(q_pos, "q_pos"), float(rope_base), float(yarn_scale), float(yarn_beta_fast),
                   float(yarn_beta_slow), _int32(prefix_len, "prefix_len"), 1 if keys_prerotated else 0)


def _window(window) -> int:
    """A window as the C interface takes it: positions are int32, so a wider one is none, as one below 1 is."""
    return int(window) if 0 < window <= _INT_MAX else 0


def _int32(x, name) -> int:
    x = int(x)
    if not _INT_MIN <= x <= _INT_MAX:
        raise ValueError("%s must fit 32 bits" % name)
    return x


def _sinks(n_sink, window) -> int:
    """Sinks of a call: none without a window."""
    if n_sink < 0:
        raise ValueError("n_sink must not be negative")
    return min(int(n_sink), _INT_MAX) if window > 0 else 0


def _prefill(q, k, v, d_r, n_sink, how, out, workspace, stream):
    """Prefill on q's device; how: arguments of _options."""
    torch = _torch or _load_torch()
    B, H_q, S_q, S_k, H_kv, d, device, pq, pk, pv = _shapes(q, k, v, d_r)
    n_sink = _sinks(n_sink, how[0])
    sizes = (B, H_q, H_kv, S_q, S_k, d)
    lib, opt = _lib or load_library(), None
    if n_sink:
        need, run, sizes, name = lib.apex_attn_sink_fwd_workspace_bytes, lib.apex_attn_sink_fwd, sizes + (d_r, n_sink), \
            "apex_attn_sink_fwd"
    elif d_r:
        need, run, sizes, name = lib.apex_attn_mla_fwd_workspace_bytes, lib.apex_attn_mla_fwd_ws, sizes + (d_r,), \
            "apex_attn_mla_fwd"
    else:
        need, run, name = lib.apex_attn_fwd_workspace_bytes, lib.apex_attn_fwd_ws, "apex_attn_fwd"
    plain = not d_r and not n_sink and _plain(how)
    if workspace is not False or not plain:
        opt = _options(*how)
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.new(q, (B, H_q, S_q, d), torch.bfloat16)
            pout = out.data_ptr()
        else:
            pout = _fit(out, "out", torch.bfloat16, (B, H_q, S_q, d), device)
        pws, size = None, need(*sizes, opt) if workspace is None else 0
        if workspace is not None and workspace is not False or size:
            ws = at.workspace(workspace, q, size)
            pws, size = ws.data_ptr(), ws.nbytes
        if plain and pws is None:
            status = lib.apex_attn_fwd(pq, pk, pv, pout, *sizes, _window(how[0]), _int32(how[1], "q_pos0"), how[2],
                                       at.handle)
        else:
            status = run(pq, pk, pv, pout, *sizes, opt, pws, size, at.handle)
        if status:
            raise ApexError(status, name)
    finally:
        at.leave()
    return out


def _decode(q, k_cache, v_cache, d_r, n_sink, how, out, workspace, stream):
    """Decode on q's device; how: arguments of _options."""
    torch = _torch or _load_torch()
    B, H_q, one, S_k, H_kv, d, device, pq, pk, pv = _shapes(q, k_cache, v_cache, d_r)
    if one != 1:
        raise ValueError("decode takes one query per sequence")
    n_sink = _sinks(n_sink, how[0])
    lib, sizes = _lib or load_library(), (B, H_q, H_kv, S_k, d)
    plain = not d_r and not n_sink and _plain(how)
    opt = None if plain else _options(*how)
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.new(q, (B, H_q, 1, d), torch.bfloat16)
            pout = out.data_ptr()
        else:
            pout = _fit(out, "out", torch.bfloat16, (B, H_q, 1, d), device)
        ws = at.workspace(workspace, q, lib.apex_attn_decode_workspace_bytes(*sizes) if workspace is None else 0)
        tail = (ws.data_ptr(), ws.nbytes, at.handle)
        if plain:
            name, status = "apex_attn_decode", lib.apex_attn_decode(
                pq, pk, pv, pout, *sizes, _window(how[0]), _int32(how[1], "q_pos"), how[2], *tail)
        elif n_sink:
            name, status = "apex_attn_sink_decode", lib.apex_attn_sink_decode(pq, pk, pv, pout, *sizes, d_r, n_sink, opt,
                                                                              *tail)
        elif d_r:
            name, status = "apex_attn_mla_decode", lib.apex_attn_mla_decode(pq, pk, pv, pout, *sizes, d_r, opt, *tail)
        else:
            name, status = "apex_attn_decode", lib.apex_attn_decode_ex(pq, pk, pv, pout, *sizes, opt, *tail)
        if status:
            raise ApexError(status, name)
    finally:
        at.leave()
    return out


def _plain(how) -> bool:
    """Whether of the arguments of _options only window, position and base count."""
    return how[3] <= 1.0 and how[6] == 0 and not how[7]


def _shapes(q, k, v, d_r):
    """Sizes of queries, keys and values, their device and addresses."""
    bf16 = _torch.bfloat16
    B, H_q, S_q, d_qk = _rows4(q, "q")
    _, H_kv, S_k, d = _rows4(v, "v")
    if max(B, H_q, S_q, H_kv, S_k, d_qk) > _INT_MAX:
        raise ValueError("more sequences, heads or tokens than are taken")
    if d_qk != d + d_r:
        raise ValueError("q must have the row length of v" + (" and d_r" if d_r else ""))
    device = q.get_device()
    return (B, H_q, S_q, S_k, H_kv, d, device, _fit(q, "q", bf16, (B, H_q, S_q, d_qk), device),
            _fit(k, "k", bf16, (B, H_kv, S_k, d_qk), device), _fit(v, "v", bf16, (B, H_kv, S_k, d), device))


def fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, *, window: int = 0, q_pos0: int = 0,
                        rope_base: float = 10000.0, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
                        yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False,
                        n_sink: int = 0) -> int:
    """Workspace bytes a prefill with these arguments uses (0: none; see apex_attn_fwd_workspace_bytes)."""
    opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                   keys_prerotated)
    n_sink = _sinks(n_sink, window)
    if n_sink:
        return int(apex_attn_sink_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, 0, n_sink, opt))
    return int(apex_attn_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, opt))


def fwd(q, k, v, *, window: int = 0, q_pos0: int = 0, rope_base: float = 10000.0, out=None, stream=None,
        yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, prefix_len: int = 0,
        keys_prerotated: bool = False, workspace=None, n_sink: int = 0):
    """Prefill. q [B,H_q,S_q,d], k/v [B,H_kv,S_k,d] (bf16, CUDA) -> out [B,H_q,S_q,d].

    n_sink: the first keys, which stay visible behind a window (sinks).

    workspace: None -- when the library would rotate the keys once before the
    prefill (fwd_workspace_bytes > 0), a buffer for them is taken from torch's
    allocator and apex_attn_fwd_ws runs; a uint8 CUDA tensor -- that buffer;
    False -- no workspace (apex_attn_fwd / apex_attn_fwd_ex)."""
    return _prefill(q, k, v, 0, n_sink, (window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow,
                                         prefix_len, keys_prerotated), out, workspace, stream)


def mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, d_r, *, window: int = 0, q_pos0: int = 0,
                            rope_base: float = 10000.0, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
                            yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False,
                            n_sink: int = 0) -> int:
    """Workspace bytes a decoupled-RoPE prefill with these arguments uses (0: none; see
    apex_attn_mla_fwd_workspace_bytes)."""
    opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                   keys_prerotated)
    n_sink = _sinks(n_sink, window)
    if n_sink:
        return int(apex_attn_sink_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, int(d_r), n_sink, opt))
    return int(apex_attn_mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, int(d_r), opt))


def mla_fwd(q, k, v, d_r: int, *, window: int = 0, q_pos0: int = 0, rope_base: float = 10000.0, out=None,
            stream=None, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0,
            prefix_len: int = 0, keys_prerotated: bool = False, workspace=None, n_sink: int = 0):
    """Decoupled-RoPE prefill. q [B,H_q,S_q,d_h+d_r], k [B,H_kv,S_k,d_h+d_r], v [B,H_kv,S_k,d_h]
    (bf16, CUDA; rows [content | rope part]) -> out [B,H_q,S_q,d_h].

    n_sink: the first keys, which stay visible behind a window (sinks).

    workspace: None -- a buffer from torch's allocator when the library would rotate
    the keys' rope parts once before the prefill (mla_fwd_workspace_bytes > 0); a
    uint8 CUDA tensor -- that buffer; False -- no workspace (apex_attn_mla_fwd)."""
    return _prefill(q, k, v, int(d_r), n_sink, (window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow,
                                                prefix_len, keys_prerotated), out, workspace, stream)


def decode_workspace_bytes(B, H_q, H_kv, S_k, d_h) -> int:
    return int(apex_attn_decode_workspace_bytes(B, H_q, H_kv, S_k, d_h))


def decode(q, k_cache, v_cache, q_pos: int, *, window: int = 0, rope_base: float = 10000.0, out=None,
           workspace=None, stream=None, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
           yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False, n_sink: int = 0):
    """Decode. q [B,H_q,1,d], caches [B,H_kv,S_k,d] (bf16, CUDA) -> out [B,H_q,1,d].

    n_sink: the first keys, which stay visible behind a window (sinks)."""
    return _decode(q, k_cache, v_cache, 0, n_sink, (window, q_pos, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow,
                                                    prefix_len, keys_prerotated), out, workspace, stream)


def mla_decode(q, k_cache, v_cache, q_pos: int, d_r: int, *, window: int = 0, rope_base: float = 10000.0,
               out=None, workspace=None, stream=None, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
               yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False,
               n_sink: int = 0):
    """Decoupled-RoPE decode. q [B,H_q,1,d_h+d_r], k_cache [B,H_kv,S_k,d_h+d_r], v_cache [B,H_kv,S_k,d_h]
    (bf16, CUDA; rows [content | rope part]) -> out [B,H_q,1,d_h].

    n_sink: the first keys, which stay visible behind a window (sinks)."""
    return _decode(q, k_cache, v_cache, int(d_r), n_sink, (window, q_pos, rope_base, yarn_scale, yarn_beta_fast,
                                                           yarn_beta_slow, prefix_len, keys_prerotated), out,
                   workspace, stream)


def rope_keys(k, *, pos0: int = 0, out=None, rope_base: float = 10000.0, yarn_scale: float = 1.0,
              yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, stream=None):
    """Rotate keys k [B,H,S,d] (bf16, CUDA) to positions pos0 + s: out = RoPE(k) (pre-rotated cache)."""
    return _turn_keys(k, None, pos0, out, (rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow), stream)


def mla_rope_keys(k, d_r: int, *, pos0: int = 0, out=None, rope_base: float = 10000.0, yarn_scale: float = 1.0,
                  yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, stream=None):
    """Decoupled-RoPE key rows k [B,H,S,d_h+d_r] (bf16, CUDA; [content | rope part]) with the
    rope part rotated to positions pos0 + s and the content part copied (pre-rotated cache)."""
    return _turn_keys(k, _int32(d_r, "d_r"), pos0, out, (rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow), stream)


def _turn_keys(k, d_r, pos0, out, freq, stream):
    """Rows of k turned, or with a d_r their last d_r entries."""
    torch = _torch or _load_torch()
    shape = B, H, S, d = _rows4(k, "k")
    device = k.get_device()
    pk = _fit(k, "k", torch.bfloat16, shape, device)
    _int32(B * H, "sequences times heads"), _int32(S, "tokens"), _int32(d, "row length")
    lib, opt, pos0 = _lib or load_library(), _options(0, 0, *freq), _int32(pos0, "pos0")
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.new(k, shape, torch.bfloat16)
        pout = _fit(out, "out", torch.bfloat16, shape, device)
        if d_r is None:
            name, status = "apex_attn_rope_keys", lib.apex_attn_rope_keys(pk, pout, B * H, S, d, pos0, S * d, S * d, opt,
                                                                          at.handle)
        else:
            name, status = "apex_attn_mla_rope_keys", lib.apex_attn_mla_rope_keys(pk, pout, B * H, S, d - d_r, d_r, pos0,
                                                                                  S * d, S * d, opt, at.handle)
        if status:
            raise ApexError(status, name)
    finally:
        at.leave()
    return out


# ------------------------------------------------------------------ over caches of rotated keys
# A decode step makes several of these calls, each a few microseconds on the device, so
# the checks of a call that is right are kept short; _refuse says what is wrong otherwise.
def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


_INT_MIN, _INT_MAX = -2 ** 31, 2 ** 31 - 1  # of the C interface: ctypes drops what does not fit


def _refuse(t, name, dtype, shape, device):
    torch = _torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError("%s must be a CUDA %s tensor" % (name, str(dtype).replace("torch.", "")))
    if t.get_device() != device:
        raise ValueError("%s is on another device than the other tensors" % name)
    raise ValueError("%s must be a contiguous tensor of shape %s" % (name, tuple(shape)))


def _fit(t, name, dtype, shape, device):
    """Address of a contiguous tensor of this dtype and shape on CUDA device `device` (>= 0)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, device)


def _rows4(t, name):
    """Shape of a 4-D bf16 CUDA tensor."""
    torch = _torch
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise TypeError("%s must be a CUDA bf16 tensor" % name)
    shape = t.shape
    if len(shape) != 4:
        raise ValueError("%s must be a 4-D tensor" % name)
    return shape


class _Launch:
    """`device` made current, and the stream to launch on: the one given, else the
    device's current stream."""
    __slots__ = ("device", "stream", "handle", "guard")

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None
        if stream is None:
            self.handle = _torch._C._cuda_getCurrentRawStream(device)
        else:
            if stream.device_index != device:
                raise ValueError("stream and tensors are on different devices")
            self.handle = stream.cuda_stream
        if _torch._C._cuda_getDevice() != device:
            self.guard = _torch.cuda.device(device)
            self.guard.__enter__()

    def leave(self):
        if self.guard is not None:
            self.guard.__exit__(None, None, None)

    def new(self, like, shape, dtype):
        """A tensor from torch's allocator: the launch stream's memory, as that of the current
        one may still be in use there, kept until the current stream is done with it too."""
        if self.stream is None:
            return _torch.empty(shape, dtype=dtype, device=like.device)
        now = _torch.cuda.current_stream(self.device)
        with _torch.cuda.stream(self.stream):
            t = _torch.empty(shape, dtype=dtype, device=like.device)
        t.record_stream(now)
        return t

    def workspace(self, given, like, need):
        if given is None:
            return self.new(like, need if need > 16 else 16, _torch.uint8)
        if not given.is_cuda or given.get_device() != self.device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the other tensors")
        return given


# apex_rope_tensor and apex_rope_options as bytes: quicker to make than ctypes structs
_ROPE_TENSOR = struct.Struct("@PPiiqqqqqq")
_ROPE_OPTIONS = struct.Struct("@iiiifffff")
assert _ROPE_TENSOR.size == ctypes.sizeof(RopeTensor) and _ROPE_OPTIONS.size == ctypes.sizeof(RopeOptions)
_rope_options = functools.lru_cache(maxsize=64)(_ROPE_OPTIONS.pack)


def _turn_options(name, layout, rot_start, d_rot, inverse, rope_base, linear_scale, yarn_scale, yarn_beta_fast,
                  yarn_beta_slow):
    """apex_rope_options as bytes."""
    if layout != "interleaved" and layout != "half":
        raise ValueError("layout must be 'interleaved' or 'half'")
    if d_rot is None:
        d_rot = 0
    elif d_rot <= 0:
        raise ValueError("d_rot must be positive")
    try:
        return _rope_options(1 if layout == "half" else 0, rot_start, d_rot, 1 if inverse else 0, rope_base,
                             linear_scale, yarn_scale, yarn_beta_fast, yarn_beta_slow)
    except struct.error as e:
        raise ValueError("%s's options: %s" % (name, e)) from None


def _row_pair(x, out, name, B, S, into, device):
    """Heads, entries and strides of a tensor and of its output."""
    bf16 = _torch.bfloat16
    try:
        known = x.dtype is bf16 and out.dtype is bf16 and x.get_device() == device == out.get_device()
    except AttributeError:
        known = False
    if not known:
        _rows4(x, name)
        _rows4(out, name + "_out")
        raise ValueError("%s or %s_out is on another device than q" % (name, name))
    xs, to = x.shape, out.shape
    if len(xs) != 4 or len(to) != 4:
        raise ValueError("%s and %s_out must be 4-D tensors" % (name, name))
    n_seq, heads, n, d = xs
    if n_seq != B or n != S:
        raise ValueError("%s must have the batch and length of q" % name)
    rows = to[2]
    if to != xs and (not into or to != (B, heads, rows, d)):
        raise ValueError("%s_out does not fit %s" % (name, name))
    if heads > _INT_MAX or d > _INT_MAX or rows > _INT_MAX:
        raise ValueError("%s has more heads or entries, or %s_out more rows, than are taken" % (name, name))
    xb, xh, xr, xe = x.stride()
    ob, oh, orow, oe = out.stride()
    if (xe != 1 or oe != 1) and d > 1:
        raise ValueError("the last dimension of %s and %s_out must be contiguous" % (name, name))
    if (ob == 0 and B > 1) or (oh == 0 and heads > 1) or (orow == 0 and rows > 1):
        raise ValueError("%s_out repeats its elements" % name)
    return heads, d, xb, xh, xr, ob, oh, orow


def _rope_rows(x, out, name, B, S, into, device):
    """apex_rope_tensor of a tensor and its output, as bytes."""
    return _ROPE_TENSOR.pack(x.data_ptr(), out.data_ptr(), *_row_pair(x, out, name, B, S, into, device))


def rope(q, k=None, v=None, *, positions, layout: str = "interleaved", rot_start: int = 0, d_rot=None,
         inverse: bool = False, rope_base: float = 10000.0, linear_scale: float = 1.0, yarn_scale: float = 1.0,
         yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, q_out=None, k_out=None, v_out=None, row0=None,
         stream=None):
    """Rotary positions. q [B,H_q,S,d], optional k [B,H_kv,S,d] and v [B,H_kv,S,d_v] (bf16, CUDA; any strides, rows
    contiguous), positions [B,S] or [S] int32 -> the rotated q, or (q, k) or (q, k, v) as given.

    layout: "interleaved" pairs (2i, 2i+1) or "half" pairs (i, i + d_rot/2) of the d_rot entries
    (None: all) from rot_start on; inverse: the opposite rotation, which is the gradient.
    q_out, k_out, v_out: outputs of any strides, else new contiguous tensors.  An output may be
    its own input (with row0: q's only) and must otherwise share no element with any input or
    other output.  row0 [B] int32: token s of k and v goes to row row0[b] + s of k_out and v_out
    (caches [B,H_kv,S_cap,d]); rows outside them are dropped, the others untouched."""
    torch = _torch or _load_torch()
    opt = _turn_options("rope", layout, rot_start, d_rot, inverse, rope_base, linear_scale, yarn_scale,
                        yarn_beta_fast, yarn_beta_slow)
    if k is None and (v is not None or k_out is not None) or v is None and v_out is not None:
        raise ValueError("k_out goes with k, and v and v_out with k")
    B, _, S, _ = _rows4(q, "q")
    if B > _INT_MAX or S > _INT_MAX:
        raise ValueError("more sequences or tokens than rope takes")
    device = q.get_device()
    at = _Launch(device, stream)
    try:
        pos = _fit(positions, "positions", torch.int32, (S,) if positions.dim() == 1 else (B, S), device)
        if q_out is None:
            q_out = at.new(q, q.shape, torch.bfloat16)
        tq, tk, tv = _rope_rows(q, q_out, "q", B, S, False, device), None, None
        into, rows, start = row0 is not None, 0, None
        if into:
            if k is None or k_out is None or (v is not None and v_out is None):
                raise ValueError("row0 needs k_out, and v_out where there is a v")
            start = _fit(row0, "row0", torch.int32, (B,), device)
        if k is not None:
            if k_out is None:
                k_out = at.new(k, k.shape, torch.bfloat16)
            tk = _rope_rows(k, k_out, "k", B, S, into, device)
        if v is not None:
            if v_out is None:
                v_out = at.new(v, v.shape, torch.bfloat16)
            tv = _rope_rows(v, v_out, "v", B, S, into, device)
        if into:
            rows = k_out.shape[2]
            if v is not None and v_out.shape[2] != rows:
                raise ValueError("k_out and v_out must have the same number of rows")
        status = (_lib or load_library()).apex_attn_rope(tq, tk, tv, B, S, pos, S if positions.dim() == 2 else 0,
                                                         start, rows, opt, at.handle)
        if status:
            raise ApexError(status, "apex_attn_rope")
    finally:
        at.leave()
    return q_out if k is None else (q_out, k_out) if v is None else (q_out, k_out, v_out)


_NORM_TENSOR = struct.Struct("@PPPPPiiiiqqqqqqqqq")
assert _NORM_TENSOR.size == ctypes.sizeof(NormTensor)


def _norm_weight(w, name, heads, d, device):
    """Address of a norm's weights, whether they are fp32 and whether each head has its own."""
    torch = _torch
    if w is None:
        return 0, 0, 0
    f32 = isinstance(w, torch.Tensor) and w.dtype is torch.float32
    if not f32 and (not isinstance(w, torch.Tensor) or w.dtype is not torch.bfloat16) or not w.is_cuda:
        raise TypeError("%s_weight must be a CUDA bfloat16 or float32 tensor" % name)
    if w.get_device() != device:
        raise ValueError("%s_weight is on another device than the other tensors" % name)
    shape = w.shape
    if shape != (d,) and shape != (heads, d) or not w.is_contiguous():
        raise ValueError("%s_weight must be a contiguous tensor of shape %s or %s" % (name, (d,), (heads, d)))
    return w.data_ptr(), 1 if f32 else 0, 1 if len(shape) == 2 else 0


def _norm_rows(x, out, weight, name, B, S, into, device):
    """apex_norm_tensor of a tensor, its output and weights, as bytes."""
    heads, d, xb, xh, xr, ob, oh, orow = _row_pair(x, out, name, B, S, into, device)
    pw, f32, per_head = _norm_weight(weight, name, heads, d, device)
    return _NORM_TENSOR.pack(x.data_ptr(), 0, out.data_ptr(), pw, 0, heads, d, f32, per_head, xb, xh, xr, 0, 0, 0, ob,
                             oh, orow)


def norm_rope(q, k=None, v=None, *, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
              layout: str = "interleaved", rot_start: int = 0, d_rot=None, rope_base: float = 10000.0,
              linear_scale: float = 1.0, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
              yarn_beta_slow: float = 1.0, q_out=None, k_out=None, v_out=None, row0=None, stream=None):
    """RMS norm of every head, then its rotary position, in one pass. q [B,H_q,S,d], optional k [B,H_kv,S,d] and
    v [B,H_kv,S,d_v] (bf16, CUDA; any strides, rows contiguous), positions [B,S] or [S] int32 -> the new q, or
    (q, k) or (q, k, v) as given.

    A row x becomes R(x / sqrt(mean(x^2) + eps) * weight): the whole row is normed, the d_rot entries from
    rot_start on are turned.  q_weight, k_weight: bf16 or fp32, [d] or, for each head its own, [H,d] (None: ones).
    Layouts, frequencies, outputs and row0 (appending k and v to caches) as for rope.  Not recorded by autograd:
    norm_rope_grad gives the gradients."""
    torch = _torch or _load_torch()
    if k is None and (v is not None or k_out is not None or k_weight is not None) or v is None and v_out is not None:
        raise ValueError("k_out and k_weight go with k, and v and v_out with k")
    B, _, S, _ = _rows4(q, "q")
    if B > _INT_MAX or S > _INT_MAX:
        raise ValueError("more sequences or tokens than norm_rope takes")
    device = q.get_device()
    opt = _turn_options("norm_rope", layout, rot_start, d_rot, False, rope_base, linear_scale, yarn_scale,
                        yarn_beta_fast, yarn_beta_slow)
    at = _Launch(device, stream)
    try:
        pos = _fit(positions, "positions", torch.int32, (S,) if positions.dim() == 1 else (B, S), device)
        if q_out is None:
            q_out = at.new(q, q.shape, torch.bfloat16)
        tq, tk, tv = _norm_rows(q, q_out, q_weight, "q", B, S, False, device), None, None
        into, rows, start = row0 is not None, 0, None
        if into:
            if k is None or k_out is None or (v is not None and v_out is None):
                raise ValueError("row0 needs k_out, and v_out where there is a v")
            start = _fit(row0, "row0", torch.int32, (B,), device)
        if k is not None:
            if k_out is None:
                k_out = at.new(k, k.shape, torch.bfloat16)
            tk = _norm_rows(k, k_out, k_weight, "k", B, S, into, device)
        if v is not None:
            if v_out is None:
                v_out = at.new(v, v.shape, torch.bfloat16)
            tv = _rope_rows(v, v_out, "v", B, S, into, device)
        if into:
            rows = k_out.shape[2]
            if v is not None and v_out.shape[2] != rows:
                raise ValueError("k_out and v_out must have the same number of rows")
        status = (_lib or load_library()).apex_attn_norm_rope(
            tq, tk, tv, B, S, pos, S if positions.dim() == 2 else 0, start, rows, opt, eps, at.handle)
        if status:
            raise ApexError(status, "apex_attn_norm_rope")
    finally:
        at.leave()
    return q_out if k is None else (q_out, k_out) if v is None else (q_out, k_out, v_out)


@functools.lru_cache(maxsize=256)
def norm_rope_grad_workspace_bytes(H_q, H_kv, d_q, d_k=None) -> int:
    """Workspace bytes of norm_rope_grad for these sizes (0: invalid; H_kv 0: without k)."""
    return int(apex_attn_norm_rope_grad_workspace_bytes(H_q, H_kv, d_q, d_q if d_k is None else d_k))


def norm_rope_grad(q_grad, q, k_grad=None, k=None, *, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                   layout: str = "interleaved", rot_start: int = 0, d_rot=None, rope_base: float = 10000.0,
                   linear_scale: float = 1.0, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
                   yarn_beta_slow: float = 1.0, q_out=None, k_out=None, workspace=None, stream=None):
    """Gradients of norm_rope. q_grad and k_grad (of its results), q and k (its inputs) and the options as given to
    it -> (gradient of q, of q_weight) or, with k, (of q, of k, of q_weight, of k_weight).

    The gradients of q and k are bf16 (q_out, k_out: where to, any strides; such an output may be its own gradient
    or input), those of the weights fp32, shaped as they (None without weights)."""
    torch = _torch or _load_torch()
    if (k is None) != (k_grad is None) or k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k, k_grad, k_out and k_weight go together")
    B, H_q, S, d_q = _rows4(q, "q")
    if B > _INT_MAX or S > _INT_MAX:
        raise ValueError("more sequences or tokens than norm_rope_grad takes")
    device = q.get_device()
    opt = _turn_options("norm_rope_grad", layout, rot_start, d_rot, False, rope_base, linear_scale, yarn_scale,
                        yarn_beta_fast, yarn_beta_slow)
    at = _Launch(device, stream)

    def rows(x, grad, out, weight, name):
        if out is None:
            out = at.new(x, x.shape, torch.bfloat16)
        heads, d, xb, xh, xr, ob, oh, orow = _row_pair(x, out, name, B, S, False, device)
        if _rows4(grad, name + "_grad") != x.shape or grad.get_device() != device:
            raise ValueError("%s_grad does not fit %s" % (name, name))
        gb, gh, gr, ge = grad.stride()
        if ge != 1 and d > 1:
            raise ValueError("the last dimension of %s_grad must be contiguous" % name)
        pw, f32, per_head = _norm_weight(weight, name, heads, d, device)
        dw = None if weight is None else at.new(weight, weight.shape, torch.float32)
        return out, dw, _NORM_TENSOR.pack(x.data_ptr(), grad.data_ptr(), out.data_ptr(), pw,
                                          0 if dw is None else dw.data_ptr(), heads, d, f32, per_head, xb, xh, xr, gb,
                                          gh, gr, ob, oh, orow)

    try:
        pos = _fit(positions, "positions", torch.int32, (S,) if positions.dim() == 1 else (B, S), device)
        q_out, q_dw, tq = rows(q, q_grad, q_out, q_weight, "q")
        tk, k_dw, H_kv, d_k = None, None, 0, 0
        if k is not None:
            _, H_kv, _, d_k = _rows4(k, "k")
            k_out, k_dw, tk = rows(k, k_grad, k_out, k_weight, "k")
        ws = at.workspace(workspace, q, norm_rope_grad_workspace_bytes(H_q, H_kv, d_q, d_k))
        status = (_lib or load_library()).apex_attn_norm_rope_grad(
            tq, tk, B, S, pos, S if positions.dim() == 2 else 0, opt, eps, ws.data_ptr(), ws.nbytes, at.handle)
        if status:
            raise ApexError(status, "apex_attn_norm_rope_grad")
    finally:
        at.leave()
    return (q_out, q_dw) if k is None else (q_out, k_out, q_dw, k_dw)


def _cache_shapes(q, k_cache, v_cache):
    """Sizes of queries and caches, their device and addresses."""
    bf16 = _torch.bfloat16
    try:
        B, H_q, T, d_qk = q.shape
        _, H_kv, S_cap, d_v = v_cache.shape
        device = q.get_device()
    except (AttributeError, ValueError):
        device = -1
    if device < 0:
        _rows4(q, "q")
        _rows4(v_cache, "v_cache")
        raise ValueError("q and v_cache must be 4-D CUDA tensors")
    return (B, H_q, T, d_qk, H_kv, S_cap, d_v, device, _fit(q, "q", bf16, (B, H_q, T, d_qk), device),
            _fit(k_cache, "k_cache", bf16, (B, H_kv, S_cap, d_qk), device),
            _fit(v_cache, "v_cache", bf16, (B, H_kv, S_cap, d_v), device))


@functools.lru_cache(maxsize=256)
def tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v=None) -> int:
    """Workspace bytes of tree_decode for these sizes (0: invalid; see apex_attn_tree_workspace_bytes)."""
    return int(apex_attn_tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_qk if d_v is None else d_v))


def tree_decode(q, k_cache, v_cache, lens, *, tree_mask=None, positions=None, window: int = 0, scale=None, out=None,
                workspace=None, stream=None, n_sink: int = 0):
    """Attention of T drafted tokens per sequence over a cache of rotated keys. q [B,H_q,T,d_qk] (rotated),
    caches [B,H_kv,S_cap,d_qk] / [B,H_kv,S_cap,d_v] with the drafts' rows at lens[b] + u, lens [B] int32
    -> out [B,H_q,T,d_v].

    tree_mask [B,T] or [T] int64: bit u of word t set when draft t sees draft u (None: u <= t);
    positions [B,T] int32: the drafts' positions, for a window (None: lens[b] + t); cached row j is
    then at position j, which is not so after evict or an append at other rows.
    n_sink: the first positions, which stay visible behind a window (sinks).
    scale: factor of the scores (None or 0: 1 / sqrt(d_qk))."""
    torch = _torch or _load_torch()
    B, H_q, T, d_qk, H_kv, S_cap, d_v, device, pq, pk, pv = _cache_shapes(q, k_cache, v_cache)
    plens = _fit(lens, "lens", torch.int32, (B,), device)
    window = _window(window)
    n_sink = _sinks(n_sink, window)
    pmask = ppos = None
    stride = 0
    if tree_mask is not None:
        one = tree_mask.dim() == 1
        pmask = _fit(tree_mask, "tree_mask", torch.int64, (T,) if one else (B, T), device)
        stride = 0 if one else T
    if positions is not None:
        ppos = _fit(positions, "positions", torch.int32, (B, T), device)
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.new(q, (B, H_q, T, d_v), torch.bfloat16)
            pout = out.data_ptr()
        else:
            pout = _fit(out, "out", torch.bfloat16, (B, H_q, T, d_v), device)
        ws = at.workspace(workspace, q, tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v))
        # the calls without sinks and with them differ by one argument
        lib, sinks = _lib or load_library(), (n_sink,) if n_sink else ()
        status = (lib.apex_attn_sink_tree_decode if n_sink else lib.apex_attn_tree_decode)(
            pq, pk, pv, pout, B, H_q, H_kv, T, S_cap, d_qk, d_v, plens, pmask, stride, ppos, window, *sinks,
            0.0 if scale is None else scale, ws.data_ptr(), ws.nbytes, at.handle)
        if status:
            raise ApexError(status, "apex_attn_tree_decode")
    finally:
        at.leave()
    return out


@functools.lru_cache(maxsize=256)
def decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_v=None) -> int:
    """Workspace bytes of decode_weights for these sizes (0: invalid)."""
    return int(apex_attn_decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_qk if d_v is None else d_v))


def decode_weights(q, k_cache, v_cache, lens, acc, *, scale=None, out=None, workspace=None, stream=None):
    """Decode over a cache of rotated keys that adds each row's attention weight to acc. q [B,H_q,1,d_qk]
    (rotated), caches [B,H_kv,S_cap,d_qk] / [B,H_kv,S_cap,d_v], lens [B] int32, acc [B,H_kv,S_cap] fp32
    (changed in place, up to lens[b]) -> out [B,H_q,1,d_v].

    scale: factor of the scores (None or 0: 1 / sqrt(d_qk))."""
    torch = _torch or _load_torch()
    B, H_q, T, d_qk, H_kv, S_cap, d_v, device, pq, pk, pv = _cache_shapes(q, k_cache, v_cache)
    if T != 1:
        raise ValueError("decode_weights takes one query per sequence")
    plens = _fit(lens, "lens", torch.int32, (B,), device)
    pacc = _fit(acc, "acc", torch.float32, (B, H_kv, S_cap), device)
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.new(q, (B, H_q, 1, d_v), torch.bfloat16)
            pout = out.data_ptr()
        else:
            pout = _fit(out, "out", torch.bfloat16, (B, H_q, 1, d_v), device)
        ws = at.workspace(workspace, q, decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_v))
        status = (_lib or load_library()).apex_attn_decode_weights(
            pq, pk, pv, pout, B, H_q, H_kv, S_cap, d_qk, d_v, plens, pacc, 0.0 if scale is None else scale,
            ws.data_ptr(), ws.nbytes, at.handle)
        if status:
            raise ApexError(status, "apex_attn_decode_weights")
    finally:
        at.leave()
    return out


@functools.lru_cache(maxsize=256)
def evict_workspace_bytes(B, H_kv, S_cap, budget) -> int:
    """Workspace bytes of evict for these sizes (0: invalid)."""
    return int(apex_attn_evict_workspace_bytes(B, H_kv, S_cap, budget))


def evict(k_cache, v_cache, acc, lens, budget: int, *, n_sink: int = 0, n_recent: int = 0, positions=None,
          next_pos=None, acc_out=None, positions_out=None, lens_out=None, workspace=None, stream=None):
    """Cut each (sequence, KV head) of a cache to `budget` rows, in place: the first n_sink and last n_recent
    positions, then the largest acc. caches [B,H_kv,S_cap,d], acc [B,H_kv,S_cap] fp32, lens [B] int32,
    positions [B,H_kv,S_cap] int32 (None: the row index), next_pos [B] int32 (None: lens, or one past
    the largest of the head's positions where that is more)
    -> (acc_out, positions_out, lens_out), in the new order of rows: row j is no longer at position j, so
    that tree_decode takes no window over the cache from then on."""
    torch = _torch or _load_torch()
    for n, x in (("budget", budget), ("n_sink", n_sink), ("n_recent", n_recent)):
        _int32(x, n)
    B, H_kv, S_cap, d_k = _rows4(k_cache, "k_cache")
    if B > _INT_MAX or H_kv > _INT_MAX or S_cap > _INT_MAX:
        raise ValueError("more sequences, heads or rows than evict takes")
    d_v = _rows4(v_cache, "v_cache")[3]
    device = k_cache.get_device()
    rows = (B, H_kv, S_cap)
    i32, f32 = torch.int32, torch.float32
    pk = _fit(k_cache, "k_cache", torch.bfloat16, (B, H_kv, S_cap, d_k), device)
    pv = _fit(v_cache, "v_cache", torch.bfloat16, (B, H_kv, S_cap, d_v), device)
    pacc = _fit(acc, "acc", f32, rows, device)
    plens = _fit(lens, "lens", i32, (B,), device)
    ppos = None if positions is None else _fit(positions, "positions", i32, rows, device)
    pnext = None if next_pos is None else _fit(next_pos, "next_pos", i32, (B,), device)
    at = _Launch(device, stream)
    try:
        if acc_out is None:
            acc_out = at.new(acc, rows, f32)
        if positions_out is None:
            positions_out = at.new(lens, rows, i32)
        if lens_out is None:
            lens_out = at.new(lens, (B,), i32)
        ws = at.workspace(workspace, acc, evict_workspace_bytes(B, H_kv, S_cap, budget))
        status = (_lib or load_library()).apex_attn_evict(
            pk, pv, B, H_kv, S_cap, d_k, d_v, pacc, ppos, plens, pnext, budget, n_sink, n_recent,
            _fit(acc_out, "acc_out", f32, rows, device), _fit(positions_out, "positions_out", i32, rows, device),
            _fit(lens_out, "lens_out", i32, (B,), device), ws.data_ptr(), ws.nbytes, at.handle)
        if status:
            raise ApexError(status, "apex_attn_evict")
    finally:
        at.leave()
    return acc_out, positions_out, lens_out


# ------------------------------------------------------------------ over caches held in 4 bits
_BITS4_TENSOR = struct.Struct("@PPPPqqqi4x")
assert _BITS4_TENSOR.size == ctypes.sizeof(Bits4Tensor)


def _packed4(x4, scales, name, like):
    """Sizes (B, H_kv, S_cap, d) and device of a packed tensor, and its addresses."""
    torch = _torch
    try:
        B, H, S_cap, half = x4.shape
        device = x4.get_device()
    except (AttributeError, ValueError):
        device = -1
    if device < 0:
        raise (ValueError if isinstance(x4, torch.Tensor) and x4.is_cuda else TypeError)(
            "%s4 must be a 4-D CUDA uint8 tensor" % name)
    if like is not None and like != (B, H, S_cap, device):
        raise ValueError("%s4 must have the batch, heads, rows and device of k4" % name)
    if max(B, H, S_cap, half) > _INT_MAX // 2:
        raise ValueError("%s4 has more sequences, heads or rows than a 4-bit cache takes" % name)
    return (B, H, S_cap, device), 2 * half, _fit(x4, name + "4", torch.uint8, (B, H, S_cap, half), device), \
        _fit(scales, name + "_scale", torch.float8_e4m3fn, (B, H, S_cap, half // 8), device)


def _factor4(f, name, H, device):
    return None if f is None else _fit(f, name + "_factor", _torch.float32, (H,), device)


def _rows4_of(x, name, B, H, S, d, device):
    """Address and strides of bf16 rows [B,H,S,d] of any strides."""
    if _rows4(x, name) != (B, H, S, d) or x.get_device() != device:
        raise ValueError("%s must be of shape %s, on the device of k4" % (name, (B, H, S, d)))
    b, h, s, e = x.stride()
    if e != 1 and d > 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return x.data_ptr(), b, h, s


def append4(k, v, k4, k_scale, v4, v_scale, *, row0=None, k_factor=None, v_factor=None, stream=None):
    """Append keys and values to a 4-bit cache, in place. k [B,H_kv,S,d_k], v [B,H_kv,S,d_v] (bf16, CUDA; any strides,
    rows contiguous) go to rows row0[b] + s (row0 [B] int32; None: s) of k4 [B,H_kv,S_cap,d_k/2], v4 (uint8: two e2m1
    values to a byte) and k_scale [B,H_kv,S_cap,d_k/16], v_scale (float8_e4m3fn: of 16 entries).

    k_factor, v_factor [H_kv] fp32 (None: 1): entries stand for value * scale * factor; best a power of two near the
    head's largest entry / 1000.  Rows outside the cache are dropped, the others untouched."""
    torch = _torch or _load_torch()
    size, d_k, pk4, pks = _packed4(k4, k_scale, "k", None)
    _, d_v, pv4, pvs = _packed4(v4, v_scale, "v", size)
    B, H, S_cap, device = size
    S = _rows4(k, "k")[2]
    if S > _INT_MAX:
        raise ValueError("more tokens than append4 takes")
    pk, kb, kh, ks = _rows4_of(k, "k", B, H, S, d_k, device)
    pv, vb, vh, vs = _rows4_of(v, "v", B, H, S, d_v, device)
    tk = _BITS4_TENSOR.pack(pk, pk4, pks, _factor4(k_factor, "k", H, device) or 0, kb, kh, ks, d_k)
    tv = _BITS4_TENSOR.pack(pv, pv4, pvs, _factor4(v_factor, "v", H, device) or 0, vb, vh, vs, d_v)
    start = None if row0 is None else _fit(row0, "row0", torch.int32, (B,), device)
    at = _Launch(device, stream)
    try:
        status = (_lib or load_library()).apex_attn_append4(tk, tv, B, H, S, S_cap, start, at.handle)
        if status:
            raise ApexError(status, "apex_attn_append4")
    finally:
        at.leave()


def unpack4(k4, k_scale, v4, v_scale, *, row0=None, n_rows=None, k_factor=None, v_factor=None, k_out=None, v_out=None,
            stream=None):
    """Rows of a 4-bit cache as bf16: row0[b] + s for s < n_rows (row0 [B] int32; None: from 0; n_rows None: S_cap)
    -> (k [B,H_kv,n_rows,d_k], v [B,H_kv,n_rows,d_v]); rows outside the cache give zeros.

    Packed tensors and factors as for append4; k_out, v_out: outputs of any strides, rows contiguous."""
    torch = _torch or _load_torch()
    size, d_k, pk4, pks = _packed4(k4, k_scale, "k", None)
    _, d_v, pv4, pvs = _packed4(v4, v_scale, "v", size)
    B, H, S_cap, device = size
    S = S_cap if n_rows is None else n_rows
    if not 0 < S <= _INT_MAX:
        raise ValueError("n_rows must be positive and fit 32 bits")
    fk, fv = _factor4(k_factor, "k", H, device), _factor4(v_factor, "v", H, device)
    start = None if row0 is None else _fit(row0, "row0", torch.int32, (B,), device)
    at = _Launch(device, stream)
    try:
        if k_out is None:
            k_out = at.new(k4, (B, H, S, d_k), torch.bfloat16)
        if v_out is None:
            v_out = at.new(v4, (B, H, S, d_v), torch.bfloat16)
        pk, kb, kh, ks = _rows4_of(k_out, "k_out", B, H, S, d_k, device)
        pv, vb, vh, vs = _rows4_of(v_out, "v_out", B, H, S, d_v, device)
        status = (_lib or load_library()).apex_attn_unpack4(
            _BITS4_TENSOR.pack(pk, pk4, pks, fk or 0, kb, kh, ks, d_k),
            _BITS4_TENSOR.pack(pv, pv4, pvs, fv or 0, vb, vh, vs, d_v), B, H, S, S_cap, start, at.handle)
        if status:
            raise ApexError(status, "apex_attn_unpack4")
    finally:
        at.leave()
    return k_out, v_out


@functools.lru_cache(maxsize=256)
def decode4_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v=None) -> int:
    """Workspace bytes of decode4 for these sizes (0: invalid; see apex_attn_decode4_workspace_bytes)."""
    return int(apex_attn_decode4_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_qk if d_v is None else d_v))


def decode4(q, k4, k_scale, v4, v_scale, lens, *, window: int = 0, n_sink: int = 0, k_factor=None, v_factor=None,
            scale=None, out=None, workspace=None, stream=None):
    """Attention of T new tokens per sequence over a 4-bit cache of rotated keys. q [B,H_q,T,d_qk] (rotated), packed
    tensors and factors as for append4 with the tokens' own rows at lens[b] + t, lens [B] int32 -> out [B,H_q,T,d_v].

    Token t sees the rows j <= lens[b] + t and, with a window > 0, of those only the last `window` and the first n_sink
    (sinks); row j is then at position j.  scale: factor of the scores (None or 0: 1 / sqrt(d_qk))."""
    torch = _torch or _load_torch()
    size, d_k, pk4, pks = _packed4(k4, k_scale, "k", None)
    _, d_v, pv4, pvs = _packed4(v4, v_scale, "v", size)
    B, H_kv, S_cap, device = size
    shape = _rows4(q, "q")
    if shape[0] != B or shape[3] != d_k:
        raise ValueError("q must have the batch and row length of k4's keys")
    _, H_q, T, d_qk = shape
    if max(H_q, T) > _INT_MAX:
        raise ValueError("more heads or tokens than decode4 takes")
    pq = _fit(q, "q", torch.bfloat16, shape, device)
    plens = _fit(lens, "lens", torch.int32, (B,), device)
    window = _window(window)
    if n_sink < 0:
        raise ValueError("n_sink must not be negative")
    fk, fv = _factor4(k_factor, "k", H_kv, device), _factor4(v_factor, "v", H_kv, device)
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.new(q, (B, H_q, T, d_v), torch.bfloat16)
            pout = out.data_ptr()
        else:
            pout = _fit(out, "out", torch.bfloat16, (B, H_q, T, d_v), device)
        ws = at.workspace(workspace, q, decode4_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v))
        status = (_lib or load_library()).apex_attn_decode4(
            pq, pk4, pks, pv4, pvs, pout, B, H_q, H_kv, T, S_cap, d_qk, d_v, plens, window, min(n_sink, S_cap), fk, fv,
            0.0 if scale is None else scale, ws.data_ptr(), ws.nbytes, at.handle)
        if status:
            raise ApexError(status, "apex_attn_decode4")
    finally:
        at.leave()
    return out
