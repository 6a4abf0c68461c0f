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
    apex_attn_rope (with RopeOptions and RopeTensor structs), apex_attn_tree_decode, apex_attn_tree_workspace_bytes,
    apex_attn_decode_weights, apex_attn_decode_weights_workspace_bytes, apex_attn_evict,
    apex_attn_evict_workspace_bytes
Tensor conveniences (torch, bf16, contiguous, on the current CUDA device):
    fwd(q, k, v, ...), decode(q, k_cache, v_cache, q_pos, ...), rope_keys(k, ...), mla_fwd(q, k, v, d_r, ...),
    mla_decode(q, k_cache, v_cache, q_pos, d_r, ...), mla_rope_keys(k, d_r, ...)
Over caches of rotated keys (int32 lengths and positions on the device; the tensors' own device):
    rope(q, k, v, positions=...), tree_decode(q, k_cache, v_cache, lens, ...),
    decode_weights(q, k_cache, v_cache, lens, acc, ...), evict(k_cache, v_cache, acc, lens, budget, ...)
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
            lib.apex_attn_tree_decode.argtypes = [vp] * 4 + [i32] * 7 + [vp, vp, i64, vp, i32, f32, vp, sz, vp]
            lib.apex_attn_tree_decode.restype = i32
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


def apex_attn_tree_decode(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens, tree_mask, mask_stride,
                          positions, window, scale, workspace, workspace_bytes, stream) -> int:
    return load_library().apex_attn_tree_decode(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens,
                                                tree_mask, mask_stride, positions, window, scale, workspace,
                                                workspace_bytes, stream)


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
def _check(t, name, ndim):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError("%s must be a CUDA bf16 tensor" % name)
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %d-D tensor" % (name, ndim))


def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _options(window=0, q_pos=0, rope_base=10000.0, yarn_scale=1.0, yarn_beta_fast=32.0, yarn_beta_slow=1.0,
             prefix_len=0, keys_prerotated=False) -> Options:
    return Options(int(window), int(q_pos), float(rope_base), float(yarn_scale), float(yarn_beta_fast),
                   float(yarn_beta_slow), int(prefix_len), 1 if keys_prerotated else 0)


def fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, *, window: int = 0, q_pos0: int = 0,
                        rope_base: float = 10000.0, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
                        yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False) -> int:
    """Workspace bytes a prefill with these arguments uses (0: none; see apex_attn_fwd_workspace_bytes)."""
    opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                   keys_prerotated)
    return int(apex_attn_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, opt))


def fwd(q, k, v, *, window: int = 0, q_pos0: int = 0, rope_base: float = 10000.0, out=None, stream=None,
        yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, prefix_len: int = 0,
        keys_prerotated: bool = False, workspace=None):
    """Prefill. q [B,H_q,S_q,d], k/v [B,H_kv,S_k,d] (bf16, CUDA) -> out [B,H_q,S_q,d].

    workspace: None -- when the library would rotate the keys once before the
    prefill (fwd_workspace_bytes > 0), a buffer for them is taken from torch's
    allocator and apex_attn_fwd_ws runs; a uint8 CUDA tensor -- that buffer;
    False -- no workspace (apex_attn_fwd / apex_attn_fwd_ex)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, 4)
    B, H_q, S_q, d = q.shape
    _, H_kv, S_k, _ = k.shape
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", 4)
    if workspace is None:
        need = fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d, window=window, q_pos0=q_pos0, rope_base=rope_base,
                                   yarn_scale=yarn_scale, yarn_beta_fast=yarn_beta_fast,
                                   yarn_beta_slow=yarn_beta_slow, prefix_len=prefix_len,
                                   keys_prerotated=keys_prerotated)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    plain = yarn_scale <= 1.0 and prefix_len == 0 and not keys_prerotated
    if workspace is not None and workspace is not False:
        opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                       keys_prerotated)
        st = apex_attn_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H_q, H_kv, S_q, S_k,
                              d, opt, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                              _stream_handle(stream))
    elif plain:
        st = apex_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H_q, H_kv, S_q, S_k, d,
                           int(window), int(q_pos0), float(rope_base), _stream_handle(stream))
    else:
        opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                       keys_prerotated)
        st = apex_attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H_q, H_kv, S_q, S_k,
                              d, opt, _stream_handle(stream))
    if st != APEX_OK:
        raise ApexError(st, "apex_attn_fwd")
    return out


def mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, d_r, *, window: int = 0, q_pos0: int = 0,
                            rope_base: float = 10000.0, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
                            yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False) -> int:
    """Workspace bytes a decoupled-RoPE prefill with these arguments uses (0: none; see
    apex_attn_mla_fwd_workspace_bytes)."""
    opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                   keys_prerotated)
    return int(apex_attn_mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, int(d_r), opt))


def mla_fwd(q, k, v, d_r: int, *, window: int = 0, q_pos0: int = 0, rope_base: float = 10000.0, out=None,
            stream=None, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0,
            prefix_len: int = 0, keys_prerotated: bool = False, workspace=None):
    """Decoupled-RoPE prefill. q [B,H_q,S_q,d_h+d_r], k [B,H_kv,S_k,d_h+d_r], v [B,H_kv,S_k,d_h]
    (bf16, CUDA; rows [content | rope part]) -> out [B,H_q,S_q,d_h].

    workspace: None -- a buffer from torch's allocator when the library would rotate
    the keys' rope parts once before the prefill (mla_fwd_workspace_bytes > 0); a
    uint8 CUDA tensor -- that buffer; False -- no workspace (apex_attn_mla_fwd)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, 4)
    B, H_q, S_q, d_qk = q.shape
    _, H_kv, S_k, d_h = v.shape
    if d_qk != d_h + d_r or k.shape[-1] != d_qk:
        raise ValueError("q / k rows must hold d_h + d_r entries")
    if out is None:
        out = torch.empty((B, H_q, S_q, d_h), dtype=torch.bfloat16, device=q.device)
    _check(out, "out", 4)
    opt = _options(window, q_pos0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                   keys_prerotated)
    if workspace is None:
        need = int(apex_attn_mla_fwd_workspace_bytes(B, H_q, H_kv, S_q, S_k, d_h, int(d_r), opt))
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None and workspace is not False:
        st = apex_attn_mla_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H_q, H_kv, S_q,
                                  S_k, d_h, int(d_r), opt, workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream_handle(stream))
        name = "apex_attn_mla_fwd_ws"
    else:
        st = apex_attn_mla_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H_q, H_kv, S_q, S_k,
                               d_h, int(d_r), opt, _stream_handle(stream))
        name = "apex_attn_mla_fwd"
    if st != APEX_OK:
        raise ApexError(st, name)
    return out


def decode_workspace_bytes(B, H_q, H_kv, S_k, d_h) -> int:
    return int(apex_attn_decode_workspace_bytes(B, H_q, H_kv, S_k, d_h))


def decode(q, k_cache, v_cache, q_pos: int, *, window: int = 0, rope_base: float = 10000.0, out=None,
           workspace=None, stream=None, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
           yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False):
    """Decode. q [B,H_q,1,d], caches [B,H_kv,S_k,d] (bf16, CUDA) -> out [B,H_q,1,d]."""
    import torch
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n, 4)
    B, H_q, one, d = q.shape
    _, H_kv, S_k, _ = k_cache.shape
    if one != 1:
        raise ValueError("decode takes one query per sequence")
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", 4)
    need = decode_workspace_bytes(B, H_q, H_kv, S_k, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    plain = yarn_scale <= 1.0 and prefix_len == 0 and not keys_prerotated
    if plain:
        st = apex_attn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), B, H_q, H_kv,
                              S_k, d, int(window), int(q_pos), float(rope_base), workspace.data_ptr(), ws_bytes,
                              _stream_handle(stream))
    else:
        opt = _options(window, q_pos, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                       keys_prerotated)
        st = apex_attn_decode_ex(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), B, H_q,
                                 H_kv, S_k, d, opt, workspace.data_ptr(), ws_bytes, _stream_handle(stream))
    if st != APEX_OK:
        raise ApexError(st, "apex_attn_decode")
    return out


def mla_decode(q, k_cache, v_cache, q_pos: int, d_r: int, *, window: int = 0, rope_base: float = 10000.0,
               out=None, workspace=None, stream=None, yarn_scale: float = 1.0, yarn_beta_fast: float = 32.0,
               yarn_beta_slow: float = 1.0, prefix_len: int = 0, keys_prerotated: bool = False):
    """Decoupled-RoPE decode. q [B,H_q,1,d_h+d_r], k_cache [B,H_kv,S_k,d_h+d_r], v_cache [B,H_kv,S_k,d_h]
    (bf16, CUDA; rows [content | rope part]) -> out [B,H_q,1,d_h]."""
    import torch
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n, 4)
    B, H_q, one, d_qk = q.shape
    _, H_kv, S_k, d_h = v_cache.shape
    if one != 1:
        raise ValueError("decode takes one query per sequence")
    if d_qk != d_h + d_r or k_cache.shape[-1] != d_qk:
        raise ValueError("q / k_cache rows must hold d_h + d_r entries")
    if out is None:
        out = torch.empty((B, H_q, 1, d_h), dtype=torch.bfloat16, device=q.device)
    _check(out, "out", 4)
    need = decode_workspace_bytes(B, H_q, H_kv, S_k, d_h)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    opt = _options(window, q_pos, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow, prefix_len,
                   keys_prerotated)
    st = apex_attn_mla_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), B, H_q, H_kv,
                              S_k, d_h, int(d_r), opt, workspace.data_ptr(), ws_bytes, _stream_handle(stream))
    if st != APEX_OK:
        raise ApexError(st, "apex_attn_mla_decode")
    return out


def rope_keys(k, *, pos0: int = 0, out=None, rope_base: float = 10000.0, yarn_scale: float = 1.0,
              yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, stream=None):
    """Rotate keys k [B,H,S,d] (bf16, CUDA) to positions pos0 + s: out = RoPE(k) (pre-rotated cache)."""
    import torch
    _check(k, "k", 4)
    B, H, S, d = k.shape
    if out is None:
        out = torch.empty_like(k)
    _check(out, "out", 4)
    if out.shape != k.shape:
        raise ValueError("out must have the shape of k")
    opt = _options(0, 0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow)
    st = apex_attn_rope_keys(k.data_ptr(), out.data_ptr(), B * H, S, d, int(pos0), S * d, S * d, opt,
                             _stream_handle(stream))
    if st != APEX_OK:
        raise ApexError(st, "apex_attn_rope_keys")
    return out


def mla_rope_keys(k, d_r: int, *, pos0: int = 0, out=None, rope_base: float = 10000.0, yarn_scale: float = 1.0,
                  yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, stream=None):
    """Decoupled-RoPE key rows k [B,H,S,d_h+d_r] (bf16, CUDA; [content | rope part]) with the
    rope part rotated to positions pos0 + s and the content part copied (pre-rotated cache)."""
    import torch
    _check(k, "k", 4)
    B, H, S, d = k.shape
    if out is None:
        out = torch.empty_like(k)
    _check(out, "out", 4)
    if out.shape != k.shape:
        raise ValueError("out must have the shape of k")
    opt = _options(0, 0, rope_base, yarn_scale, yarn_beta_fast, yarn_beta_slow)
    st = apex_attn_mla_rope_keys(k.data_ptr(), out.data_ptr(), B * H, S, d - int(d_r), int(d_r), int(pos0), S * d,
                                 S * d, opt, _stream_handle(stream))
    if st != APEX_OK:
        raise ApexError(st, "apex_attn_mla_rope_keys")
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


def _rope_rows(x, out, name, B, S, into, device):
    """apex_rope_tensor of a tensor and its output, as bytes."""
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
    if xs[0] != B or xs[2] != S:
        raise ValueError("%s must have the batch and length of q" % name)
    if (to != xs and not into) or to[0] != B or to[1] != xs[1] or to[3] != xs[3]:
        raise ValueError("%s_out does not fit %s" % (name, name))
    if xs[1] > _INT_MAX or xs[3] > _INT_MAX or to[2] > _INT_MAX:
        raise ValueError("%s has more heads or entries, or %s_out more rows, than rope takes" % (name, name))
    xb, xh, xr, xe = x.stride()
    ob, oh, orow, oe = out.stride()
    if (xe != 1 or oe != 1) and xs[3] > 1:
        raise ValueError("the last dimension of %s and %s_out must be contiguous" % (name, name))
    if (ob == 0 and B > 1) or (oh == 0 and to[1] > 1) or (orow == 0 and to[2] > 1):
        raise ValueError("%s_out repeats its elements" % name)
    return _ROPE_TENSOR.pack(x.data_ptr(), out.data_ptr(), xs[1], xs[3], xb, xh, xr, ob, oh, orow)


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
    if layout != "interleaved" and layout != "half":
        raise ValueError("layout must be 'interleaved' or 'half'")
    if d_rot is None:
        d_rot = 0
    elif d_rot <= 0:
        raise ValueError("d_rot must be positive")
    if k is None and (v is not None or k_out is not None) or v is None and v_out is not None:
        raise ValueError("k_out goes with k, and v and v_out with k")
    B, _, S, _ = _rows4(q, "q")
    if B > _INT_MAX or S > _INT_MAX:
        raise ValueError("more sequences or tokens than rope takes")
    device = q.get_device()
    try:
        opt = _rope_options(1 if layout == "half" else 0, rot_start, d_rot, 1 if inverse else 0, rope_base,
                            linear_scale, yarn_scale, yarn_beta_fast, yarn_beta_slow)
    except struct.error as e:
        raise ValueError("rope's options: %s" % e) from None
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
                workspace=None, stream=None):
    """Attention of T drafted tokens per sequence over a cache of rotated keys. q [B,H_q,T,d_qk] (rotated),
    caches [B,H_kv,S_cap,d_qk] / [B,H_kv,S_cap,d_v] with the drafts' rows at lens[b] + u, lens [B] int32
    -> out [B,H_q,T,d_v].

    tree_mask [B,T] or [T] int64: bit u of word t set when draft t sees draft u (None: u <= t);
    positions [B,T] int32: the drafts' positions, for a window (None: lens[b] + t); cached row j is
    then at position j, which is not so after evict or an append at other rows.
    scale: factor of the scores (None or 0: 1 / sqrt(d_qk))."""
    torch = _torch or _load_torch()
    B, H_q, T, d_qk, H_kv, S_cap, d_v, device, pq, pk, pv = _cache_shapes(q, k_cache, v_cache)
    plens = _fit(lens, "lens", torch.int32, (B,), device)
    if not 0 < window <= _INT_MAX:  # positions are int32: a wider window is none
        window = 0
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
        status = (_lib or load_library()).apex_attn_tree_decode(
            pq, pk, pv, pout, B, H_q, H_kv, T, S_cap, d_qk, d_v, plens, pmask, stride, ppos, window,
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
        if not _INT_MIN <= x <= _INT_MAX:
            raise ValueError("%s must fit 32 bits" % n)
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
