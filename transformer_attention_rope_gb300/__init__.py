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
import os
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
            i64, rt = ctypes.c_longlong, ctypes.POINTER(RopeTensor)
            lib.apex_attn_rope.argtypes = [rt, rt, rt, i32, i32, vp, i64, vp, i32, ctypes.POINTER(RopeOptions), vp]
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
    ref = [ctypes.byref(t) if t is not None else None for t in (q, k, v, opt)]
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
def _check_on(t, name, like, dtype, shape):
    """A contiguous tensor of this dtype and shape on the device of `like`."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError("%s must be a CUDA %s tensor" % (name, str(dtype).replace("torch.", "")))
    if t.device != like.device:
        raise ValueError("%s is on another device than the other tensors" % name)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s" % (name, tuple(shape)))


class _Launch:
    """The device of a tensor made current, and the stream to launch on: the one
    given, else that device's current stream.  Scratch taken from torch's allocator
    is kept until the stream is done with it."""

    def __init__(self, like, stream):
        import torch
        self.device = like.device
        self.guard = torch.cuda.device(like.device)
        self.given = stream
        if stream is not None and stream.device != like.device:
            raise ValueError("stream and tensors are on different devices")

    def __enter__(self):
        import torch
        self.guard.__enter__()
        self.stream = self.given if self.given is not None else torch.cuda.current_stream()
        self.handle = self.stream.cuda_stream
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)

    def workspace(self, given, need):
        """(pointer, bytes) of the caller's workspace, or of scratch of `need` bytes."""
        import torch
        if given is None:
            given = torch.empty(max(int(need), 16), dtype=torch.uint8, device=self.device)
            if self.given is not None:
                given.record_stream(self.stream)
        elif not given.is_cuda or given.device != self.device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the other tensors")
        return given.data_ptr(), given.numel() * given.element_size()


def _done(status, what):
    if status != APEX_OK:
        raise ApexError(status, what)


def _rope_rows(x, out, name, like):
    import torch
    for t, n in ((x, name), (out, name + "_out")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError("%s must be a CUDA bf16 tensor" % n)
        if t.device != like.device:
            raise ValueError("%s is on another device than the other tensors" % n)
        if t.dim() != 4 or (t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError("%s must be a 4-D tensor whose last dimension is contiguous" % n)
    if any(n > 1 and st == 0 for n, st in zip(out.shape, out.stride())):
        raise ValueError("%s_out repeats its elements" % name)
    return RopeTensor(x.data_ptr(), out.data_ptr(), x.shape[1], x.shape[3], x.stride(0), x.stride(1), x.stride(2),
                      out.stride(0), out.stride(1), out.stride(2))


def rope(q, k=None, v=None, *, positions, layout: str = "interleaved", rot_start: int = 0, d_rot=None,
         inverse: bool = False, rope_base: float = 10000.0, linear_scale: float = 1.0, yarn_scale: float = 1.0,
         yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, q_out=None, k_out=None, v_out=None, row0=None,
         stream=None):
    """Rotary positions. q [B,H_q,S,d], optional k [B,H_kv,S,d] and v [B,H_kv,S,d_v] (bf16, CUDA; any strides, rows
    contiguous), positions [B,S] or [S] int32 -> the rotated q, or (q, k) or (q, k, v) as given.

    layout: "interleaved" pairs (2i, 2i+1) or "half" pairs (i, i + d_rot/2) of the d_rot entries
    (None: all) from rot_start on; inverse: the opposite rotation, which is the gradient.
    q_out, k_out, v_out: outputs of any strides, the inputs themselves among them; else new
    contiguous tensors.  row0 [B] int32: token s of k and v goes to row row0[b] + s of k_out
    and v_out (caches [B,H_kv,S_cap,d]); rows outside them are dropped, the others untouched."""
    import torch
    if layout not in ("interleaved", "half"):
        raise ValueError("layout must be 'interleaved' or 'half'")
    if v is not None and k is None:
        raise ValueError("v goes with k")
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D tensor")
    B, _, S, _ = q.shape
    tensors, outs, out_rows = [], [], 0
    for x, o, name in ((q, q_out, "q"), (k, k_out, "k"), (v, v_out, "v")):
        if x is None:
            if o is not None:
                raise ValueError("%s_out without %s" % (name, name))
            continue
        if o is None:
            if row0 is not None and name != "q":
                raise ValueError("row0 needs %s_out" % name)
            o = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        tensors.append(_rope_rows(x, o, name, q))
        if x.shape[0] != B or x.shape[2] != S:
            raise ValueError("%s must have the batch and length of q" % name)
        into = row0 is not None and name != "q"
        if o.shape[:2] != x.shape[:2] or o.shape[3] != x.shape[3] or (o.shape[2] != S and not into):
            raise ValueError("%s_out does not fit %s" % (name, name))
        if into:
            if out_rows not in (0, o.shape[2]):
                raise ValueError("k_out and v_out must have the same number of rows")
            out_rows = o.shape[2]
        outs.append(o)
    _check_on(positions, "positions", q, torch.int32, (S,) if positions.dim() == 1 else (B, S))
    if row0 is not None:
        _check_on(row0, "row0", q, torch.int32, (B,))
    opt = RopeOptions(1 if layout == "half" else 0, int(rot_start), 0 if d_rot is None else int(d_rot),
                      1 if inverse else 0, float(rope_base), float(linear_scale), float(yarn_scale),
                      float(yarn_beta_fast), float(yarn_beta_slow))
    if d_rot is not None and int(d_rot) <= 0:
        raise ValueError("d_rot must be positive")
    with _Launch(q, stream) as at:
        tensors += [None] * (3 - len(tensors))
        _done(apex_attn_rope(tensors[0], tensors[1], tensors[2], B, S, positions.data_ptr(),
                             S if positions.dim() == 2 else 0, row0.data_ptr() if row0 is not None else None,
                             out_rows, opt, at.handle), "apex_attn_rope")
    return outs[0] if len(outs) == 1 else tuple(outs)


def _cache_shapes(q, k_cache, v_cache):
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n, 4)
    B, H_q, T, d_qk = q.shape
    _, H_kv, S_cap, d_v = v_cache.shape
    if tuple(k_cache.shape) != (B, H_kv, S_cap, d_qk) or v_cache.shape[0] != B:
        raise ValueError("k_cache / v_cache must be [B, H_kv, S_cap, d] with the batch and row length of q")
    if k_cache.device != q.device or v_cache.device != q.device:
        raise ValueError("q, k_cache and v_cache must be on one device")
    return B, H_q, T, d_qk, H_kv, S_cap, d_v


def tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v=None) -> int:
    return int(apex_attn_tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_qk if d_v is None else d_v))


def tree_decode(q, k_cache, v_cache, lens, *, tree_mask=None, positions=None, window: int = 0, scale=None, out=None,
                workspace=None, stream=None):
    """Attention of T drafted tokens per sequence over a cache of rotated keys. q [B,H_q,T,d_qk] (rotated),
    caches [B,H_kv,S_cap,d_qk] / [B,H_kv,S_cap,d_v] with the drafts' rows at lens[b] + u, lens [B] int32
    -> out [B,H_q,T,d_v].

    tree_mask [B,T] or [T] int64: bit u of word t set when draft t sees draft u (None: u <= t);
    positions [B,T] int32: the drafts' positions, for a window (None: lens[b] + t)."""
    import torch
    B, H_q, T, d_qk, H_kv, S_cap, d_v = _cache_shapes(q, k_cache, v_cache)
    _check_on(lens, "lens", q, torch.int32, (B,))
    if tree_mask is not None:
        _check_on(tree_mask, "tree_mask", q, torch.int64, (T,) if tree_mask.dim() == 1 else (B, T))
    if positions is not None:
        _check_on(positions, "positions", q, torch.int32, (B, T))
    with _Launch(q, stream) as at:
        if out is None:
            out = torch.empty((B, H_q, T, d_v), dtype=torch.bfloat16, device=q.device)
        _check_on(out, "out", q, torch.bfloat16, (B, H_q, T, d_v))
        ws, ws_bytes = at.workspace(workspace, tree_workspace_bytes(B, H_q, H_kv, T, S_cap, d_qk, d_v))
        _done(apex_attn_tree_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), B, H_q,
                                    H_kv, T, S_cap, d_qk, d_v, lens.data_ptr(),
                                    tree_mask.data_ptr() if tree_mask is not None else None,
                                    T if tree_mask is not None and tree_mask.dim() == 2 else 0,
                                    positions.data_ptr() if positions is not None else None, int(window),
                                    0.0 if scale is None else float(scale), ws, ws_bytes, at.handle),
              "apex_attn_tree_decode")
    return out


def decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_v=None) -> int:
    return int(apex_attn_decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_qk if d_v is None else d_v))


def decode_weights(q, k_cache, v_cache, lens, acc, *, scale=None, out=None, workspace=None, stream=None):
    """Decode over a cache of rotated keys that adds each row's attention weight to acc. q [B,H_q,1,d_qk]
    (rotated), caches [B,H_kv,S_cap,d_qk] / [B,H_kv,S_cap,d_v], lens [B] int32, acc [B,H_kv,S_cap] fp32
    (changed in place, up to lens[b]) -> out [B,H_q,1,d_v]."""
    import torch
    B, H_q, T, d_qk, H_kv, S_cap, d_v = _cache_shapes(q, k_cache, v_cache)
    if T != 1:
        raise ValueError("decode_weights takes one query per sequence")
    _check_on(lens, "lens", q, torch.int32, (B,))
    _check_on(acc, "acc", q, torch.float32, (B, H_kv, S_cap))
    with _Launch(q, stream) as at:
        if out is None:
            out = torch.empty((B, H_q, 1, d_v), dtype=torch.bfloat16, device=q.device)
        _check_on(out, "out", q, torch.bfloat16, (B, H_q, 1, d_v))
        ws, ws_bytes = at.workspace(workspace, decode_weights_workspace_bytes(B, H_q, H_kv, S_cap, d_qk, d_v))
        _done(apex_attn_decode_weights(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), B, H_q,
                                       H_kv, S_cap, d_qk, d_v, lens.data_ptr(), acc.data_ptr(),
                                       0.0 if scale is None else float(scale), ws, ws_bytes, at.handle),
              "apex_attn_decode_weights")
    return out


def evict_workspace_bytes(B, H_kv, S_cap, budget) -> int:
    return int(apex_attn_evict_workspace_bytes(B, H_kv, S_cap, budget))


def evict(k_cache, v_cache, acc, lens, budget: int, *, n_sink: int = 0, n_recent: int = 0, positions=None,
          next_pos=None, acc_out=None, positions_out=None, lens_out=None, workspace=None, stream=None):
    """Cut each (sequence, KV head) of a cache to `budget` rows, in place: the first n_sink and last n_recent
    positions, then the largest acc. caches [B,H_kv,S_cap,d], acc [B,H_kv,S_cap] fp32, lens [B] int32,
    positions [B,H_kv,S_cap] int32 (None: the row index), next_pos [B] int32 (None: lens)
    -> (acc_out, positions_out, lens_out), in the new order of rows."""
    import torch
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, n, 4)
    B, H_kv, S_cap, d_k = k_cache.shape
    d_v = v_cache.shape[-1]
    if tuple(v_cache.shape[:3]) != (B, H_kv, S_cap) or v_cache.device != k_cache.device:
        raise ValueError("k_cache and v_cache must hold the same rows on one device")
    at_rows = (B, H_kv, S_cap)
    _check_on(acc, "acc", k_cache, torch.float32, at_rows)
    _check_on(lens, "lens", k_cache, torch.int32, (B,))
    if positions is not None:
        _check_on(positions, "positions", k_cache, torch.int32, at_rows)
    if next_pos is not None:
        _check_on(next_pos, "next_pos", k_cache, torch.int32, (B,))
    with _Launch(k_cache, stream) as at:
        if acc_out is None:
            acc_out = torch.empty_like(acc)
        if positions_out is None:
            positions_out = torch.empty(at_rows, dtype=torch.int32, device=k_cache.device)
        if lens_out is None:
            lens_out = torch.empty_like(lens)
        _check_on(acc_out, "acc_out", k_cache, torch.float32, at_rows)
        _check_on(positions_out, "positions_out", k_cache, torch.int32, at_rows)
        _check_on(lens_out, "lens_out", k_cache, torch.int32, (B,))
        ws, ws_bytes = at.workspace(workspace, evict_workspace_bytes(B, H_kv, S_cap, int(budget)))
        _done(apex_attn_evict(k_cache.data_ptr(), v_cache.data_ptr(), B, H_kv, S_cap, d_k, d_v, acc.data_ptr(),
                              positions.data_ptr() if positions is not None else None, lens.data_ptr(),
                              next_pos.data_ptr() if next_pos is not None else None, int(budget), int(n_sink),
                              int(n_recent), acc_out.data_ptr(), positions_out.data_ptr(), lens_out.data_ptr(), ws,
                              ws_bytes, at.handle), "apex_attn_evict")
    return acc_out, positions_out, lens_out
