"""ctypes binding of libgla (include/gla.h), with the C ABI's names.

Argument marshalling only: every step of the mixer runs in libgla's CUDA
kernels. PyTorch supplies device memory and the current stream; the
functions below read shapes from the tensors, allocate outputs that the
caller did not pass, and forward raw device pointers. There is no CPU path:
if libgla.so is missing or a call fails, a GlaError is raised.

Functions:
  gla_chunk_fwd(q, k, v, log_lambda, h0=None, scale=None, chunk=128, ...) -> (o, hT)
  gla_chunk_fwd_noalloc(...)                                              -> (o, hT)
  gla_chunk_fwd_varlen(q, k, v, log_lambda, cu_seqlens, state_pool, ...)  -> o  (pool updated)
  gla_chunk_fwd_varlen_gated(q, k, v, g, cu_seqlens, state_pool, ...)     -> o  (pool updated) per-token decay
  gla_chunk_fwd_mixer(q, k, v, g, log_lambda, ...)                        -> (z, hT)
  gla_chunk_fwd_gated(q, k, v, g, h0=None, scale=None, chunk=128, ...)    -> (o, hT)  per-token decay
  gla_chunk_bwd(q, k, v, log_lambda, do, h0=None, dhT=None, ...)          -> (dq, dk, dv, dh0)
  gla_chunk_bwd_gated(q, k, v, g, do, h0=None, dhT=None, ...)             -> (dq, dk, dv, dh0, dg)
  gla_decode_step(q, k, v, log_lambda, S, scale=None, ...)                -> o  (S updated in place)
  gla_decode_step_mixer(q, k, v, log_lambda, S, g, ...)                   -> z  (S updated in place)
  gla_decode_step_gated(q, k, v, g, S, scale=None, ...)                   -> o  (S updated in place)
  gla_mixer_epilogue(o, q, k, v, g, aug=None, norm_w=None, eps=1e-6)      -> z
  gla_conv1d_fwd(x, w, b=None, win_in=None, ...)                          -> (y, win_out)
  gla_conv1d_varlen(x, w, b, cu_seqlens, win_pool, slots=None)            -> y  (pool updated)
  gla_conv1d_step(x, w, b, win)                                           -> y  (window updated)
  gla_ssm_fwd(x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, h0=None) -> (y, hT)  selective scan
  gla_ssm_varlen(x, dt, A, Bm, Cm, cu_seqlens, state_pool, ...)           -> y  (pools updated)
  gla_ssm_step(x, dt, A, Bm, Cm, state_pool, ...)                         -> y  (pools updated)
  gla_ssm_bwd(x, dt, A, Bm, Cm, dy, skip=None, z=None, ...)               -> (dx, ddt, dA, dB, dC, dskip, dz, ddt_bias, dh0)
  gla_conv1d_bwd(x, w, b, dy, win_in=None)                                -> (dx, dw, db)
  gla_rmsnorm(x, w=None, res=None, eps=1e-6)                              -> (y, s)  s = x + res
  gla_rmsnorm_q8(x, w=None, res=None, eps=1e-6, group=128)                -> (y8 e4m3, scale, s)
  gla_rmsnorm_bwd(s, w, dy, ds=None, eps=1e-6)                            -> (dx, dw)
  gla_layernorm(x, w=None, b=None, res=None, eps=1e-6)                    -> (y, s)  s = x + res
  gla_layernorm_bwd(s, w, dy, ds=None, eps=1e-6)                          -> (dx, dw, db)
  gla_tree_fwd(q, k, v, log_lambda, cu_nodes, parents, state_pool, ...)   -> o  drafted trees, the pool only read
  gla_tree_fwd_gated(q, k, v, g, cu_nodes, parents, state_pool, ...)      -> o  per-token decay
  gla_tree_commit(k, v, log_lambda, cu_nodes, parents, last, state_pool, ...) -> state_pool  (pools updated)
  gla_tree_commit_gated(k, v, g, cu_nodes, parents, last, state_pool, ...)    -> state_pool  (pools updated)
  gla_conv1d_tree(x, w, b, cu_nodes, parents, win_pool, slots=None)       -> y  the windows only read
  gla_pages_copy(pools, src, dst), gla_pages_clear(pools, slots)          (pools updated)
  gla_pages_compact(pools, live)                                          -> (map, count)  (pools updated)
  gla_check(stream=None), gla_status_string(code), gla_version()
  gla_chunk_fwd_workspace_size(...), gla_chunk_bwd_workspace_size(...)
`lib()` returns the loaded ctypes library for callers that hold raw pointers.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_lib", "libgla.so")

GLA_OK, GLA_ERR_INVALID_ARG, GLA_ERR_UNSUPPORTED, GLA_ERR_CUDA, GLA_ERR_TIMEOUT, GLA_ERR_WORKSPACE = range(6)
GLA_BF16, GLA_FP32 = 0, 1

# The public entry points declared in include/gla.h.
ABI_FUNCTIONS = ("gla_chunk_fwd", "gla_chunk_fwd_workspace_size", "gla_chunk_fwd_noalloc", "gla_chunk_fwd_varlen", "gla_chunk_fwd_varlen_gated",
                 "gla_chunk_fwd_mixer", "gla_chunk_fwd_gated", "gla_chunk_fwd_gated_workspace_size", "gla_decode_step_gated", "gla_chunk_bwd",
                 "gla_chunk_bwd_workspace_size", "gla_chunk_bwd_gated", "gla_chunk_bwd_gated_workspace_size", "gla_decode_step", "gla_decode_step_mixer", "gla_mixer_epilogue",
                 "gla_conv1d_fwd", "gla_conv1d_varlen", "gla_conv1d_step", "gla_ssm_fwd", "gla_ssm_fwd_workspace_size",
                 "gla_ssm_varlen", "gla_ssm_varlen_workspace_size", "gla_ssm_step",
                 "gla_ssm_bwd", "gla_ssm_bwd_workspace_size",
                 "gla_conv1d_bwd", "gla_conv1d_bwd_workspace_size", "gla_rmsnorm_fwd", "gla_rmsnorm_bwd",
                 "gla_rmsnorm_bwd_workspace_size", "gla_tree_fwd", "gla_tree_fwd_gated", "gla_tree_commit",
                 "gla_tree_commit_gated", "gla_conv1d_tree", "gla_pages_copy", "gla_pages_clear", "gla_pages_compact",
                 "gla_pages_compact_workspace_size", "gla_layernorm_fwd", "gla_layernorm_bwd",
                 "gla_layernorm_bwd_workspace_size", "gla_selftest_wait_timeout", "gla_check",
                 "gla_status_string", "gla_last_error", "gla_last_launch_count", "gla_version")


class GlaError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str = ""):
        self.status = status
        name = _status_name(status)
        super().__init__(f"{func} failed: {name}" + (f" -- {detail}" if detail else ""))


_lock = threading.Lock()
_lib = None
_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_ll = ctypes.c_int64


def lib():
    """Load libgla.so (built in-tree by linear_attention_chunk_gb300.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise GlaError(GLA_ERR_CUDA, "load",
                               f"{LIB_PATH} is not built; run `python -m linear_attention_chunk_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            L.gla_chunk_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i, _i, _i,
                                        _vp, _vp, _vp, _sz, _vp]
            L.gla_chunk_fwd.restype = _i
            L.gla_chunk_fwd_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i, _i, _i,
                                                _vp, _vp, _vp]
            L.gla_chunk_fwd_noalloc.restype = _i
            L.gla_chunk_fwd_varlen.argtypes = [_vp, _vp, _vp, _vp, _f, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                               _i, _i, _vp, _vp]
            L.gla_chunk_fwd_varlen.restype = _i
            L.gla_chunk_fwd_mixer.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _f, _i, _i, _i, _i, _i, _i,
                                              _i, _vp, _vp, _vp, _sz, _vp]
            L.gla_chunk_fwd_mixer.restype = _i
            L.gla_chunk_fwd_varlen_gated.argtypes = [_vp, _vp, _vp, _vp, _f, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                                     _i, _i, _i, _vp, _vp]
            L.gla_chunk_fwd_varlen_gated.restype = _i
            L.gla_chunk_fwd_gated.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                              _vp, _sz, _vp]
            L.gla_chunk_fwd_gated.restype = _i
            L.gla_chunk_fwd_gated_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
            L.gla_chunk_fwd_gated_workspace_size.restype = _sz
            L.gla_decode_step_gated.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i, _vp, _vp]
            L.gla_decode_step_gated.restype = _i
            L.gla_chunk_fwd_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
            L.gla_chunk_fwd_workspace_size.restype = _sz
            L.gla_chunk_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp]
            L.gla_chunk_bwd.restype = _i
            L.gla_chunk_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
            L.gla_chunk_bwd_workspace_size.restype = _sz
            L.gla_chunk_bwd_gated.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                              _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
            L.gla_chunk_bwd_gated.restype = _i
            L.gla_chunk_bwd_gated_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
            L.gla_chunk_bwd_gated_workspace_size.restype = _sz
            L.gla_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i, _vp, _vp]
            L.gla_decode_step.restype = _i
            L.gla_decode_step_mixer.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i,
                                                _vp, _vp]
            L.gla_decode_step_mixer.restype = _i
            L.gla_mixer_epilogue.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i, _i, _vp, _vp]
            L.gla_mixer_epilogue.restype = _i
            L.gla_conv1d_fwd.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp]
            L.gla_conv1d_fwd.restype = _i
            L.gla_conv1d_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp]
            L.gla_conv1d_varlen.restype = _i
            L.gla_conv1d_step.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp]
            L.gla_conv1d_step.restype = _i
            rows = [_vp, _ll, _vp, _ll, _vp, _vp, _ll, _vp, _ll, _vp, _vp, _ll, _vp, _i]   # x .. softplus
            L.gla_ssm_fwd.argtypes = rows + [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]
            L.gla_ssm_fwd.restype = _i
            L.gla_ssm_fwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
            L.gla_ssm_fwd_workspace_size.restype = _sz
            L.gla_ssm_varlen.argtypes = rows + [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _sz,
                                                _vp]
            L.gla_ssm_varlen.restype = _i
            L.gla_ssm_varlen_workspace_size.argtypes = [_i, _i, _i, _i, _i]
            L.gla_ssm_varlen_workspace_size.restype = _sz
            L.gla_ssm_step.argtypes = rows + [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp]
            L.gla_ssm_step.restype = _i
            L.gla_ssm_bwd.argtypes = rows + [_vp, _vp, _ll, _vp, _i, _i, _i, _i, _i] + [_vp] * 10 + [_sz, _vp]
            L.gla_ssm_bwd.restype = _i
            L.gla_ssm_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
            L.gla_ssm_bwd_workspace_size.restype = _sz
            L.gla_conv1d_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]
            L.gla_conv1d_bwd.restype = _i
            L.gla_conv1d_bwd_workspace_size.argtypes = [_i, _i, _i, _i]
            L.gla_conv1d_bwd_workspace_size.restype = _sz
            L.gla_rmsnorm_fwd.argtypes = [_vp, _vp, _vp, _f, _ll, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]
            L.gla_rmsnorm_fwd.restype = _i
            L.gla_rmsnorm_bwd.argtypes = [_vp, _vp, _vp, _vp, _f, _ll, _i, _i, _vp, _vp, _vp, _sz, _vp]
            L.gla_rmsnorm_bwd.restype = _i
            L.gla_rmsnorm_bwd_workspace_size.argtypes = [_ll, _i, _i]
            L.gla_rmsnorm_bwd_workspace_size.restype = _sz
            heads = [_vp, _ll]
            for name in ("gla_tree_fwd", "gla_tree_fwd_gated"):
                f = getattr(L, name)
                f.argtypes = heads * 3 + [_vp, _f, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp]
                f.restype = _i
            for name in ("gla_tree_commit", "gla_tree_commit_gated"):
                f = getattr(L, name)
                f.argtypes = heads * 2 + [_vp] * 6 + heads + [_vp] + [_i] * 8 + [_vp]
                f.restype = _i
            L.gla_conv1d_tree.argtypes = heads + [_vp] * 6 + [_i] * 5 + [_vp, _vp]
            L.gla_conv1d_tree.restype = _i
            pools = [ctypes.POINTER(_vp), ctypes.POINTER(_ll), _i, _i]
            L.gla_pages_copy.argtypes = pools + [_vp, _vp, _i, _vp]
            L.gla_pages_copy.restype = _i
            L.gla_pages_clear.argtypes = pools + [_vp, _i, _vp]
            L.gla_pages_clear.restype = _i
            L.gla_pages_compact.argtypes = pools + [_vp, _vp, _vp, _vp, _sz, _vp]
            L.gla_pages_compact.restype = _i
            L.gla_pages_compact_workspace_size.argtypes = [_i]
            L.gla_pages_compact_workspace_size.restype = _sz
            L.gla_layernorm_fwd.argtypes = [_vp, _vp, _vp, _vp, _f, _ll, _i, _i, _vp, _vp, _vp]
            L.gla_layernorm_fwd.restype = _i
            L.gla_layernorm_bwd.argtypes = [_vp, _vp, _vp, _vp, _f, _ll, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]
            L.gla_layernorm_bwd.restype = _i
            L.gla_layernorm_bwd_workspace_size.argtypes = [_ll, _i, _i]
            L.gla_layernorm_bwd_workspace_size.restype = _sz
            L.gla_selftest_wait_timeout.argtypes = [ctypes.c_uint, _vp, _vp]
            L.gla_selftest_wait_timeout.restype = _i
            L.gla_check.argtypes = [_vp]
            L.gla_check.restype = _i
            L.gla_status_string.argtypes = [_i]
            L.gla_status_string.restype = ctypes.c_char_p
            L.gla_last_error.argtypes = []
            L.gla_last_error.restype = ctypes.c_char_p
            L.gla_last_launch_count.argtypes = []
            L.gla_last_launch_count.restype = _i
            L.gla_version.argtypes = []
            L.gla_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _status_name(status: int) -> str:
    if _lib is None and not os.path.exists(LIB_PATH):   # that error itself: lib() holds its lock and would only repeat it
        return f"status {status}"
    try:
        return lib().gla_status_string(int(status)).decode()
    except Exception:
        return f"status {status}"


def _raise_on(status: int, func: str):
    if status != GLA_OK:
        raise GlaError(status, func, lib().gla_last_error().decode(errors="replace"))


def gla_status_string(status: int) -> str:
    return lib().gla_status_string(int(status)).decode()


def gla_version() -> str:
    return lib().gla_version().decode()


def gla_last_launch_count() -> int:
    """Kernels launched by the last entry-point call on this thread."""
    return int(lib().gla_last_launch_count())


# ------------------------------------------------------------------ helpers
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return GLA_BF16
    if t.dtype == torch.float32:
        return GLA_FP32
    raise GlaError(GLA_ERR_INVALID_ARG, "dtype", f"unsupported tensor dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", "tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", "tensors must be contiguous")
    return t.data_ptr()


def _f32(t, shape, name):
    """Pointer of an fp32 argument (decays, states), after checking its dtype
    and shape: the C ABI reads these buffers as float without knowing them."""
    if t is None:
        return None
    torch = _torch()
    if t.dtype != torch.float32:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} must be float32, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _ptr(t)


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# --------------------------------------------------------------- entry points
def gla_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk=128, dtype=GLA_BF16) -> int:
    return int(lib().gla_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, dtype))


def gla_chunk_bwd_workspace_size(B, T, H, dk, dv, chunk=128, dtype=GLA_BF16) -> int:
    return int(lib().gla_chunk_bwd_workspace_size(B, T, H, dk, dv, chunk, dtype))


def gla_chunk_fwd(q, k, v, log_lambda, h0=None, scale=None, chunk=128, *, o=None, hT=None,
                  want_hT=True, workspace=None, stream=None):
    """Chunked forward. q, k [B,T,H,dk], v [B,T,H,dv] (bf16 or fp32, CUDA),
    log_lambda [H] fp32, h0 [B,H,dk,dv] fp32 or None. Returns (o, hT)."""
    torch = _torch()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if hT is None and want_hT:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ws_need = gla_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gla_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _f32(log_lambda, (H,), "log_lambda"),
                             _f32(h0, (B, H, dk, dv), "h0"), float(scale),
                             B, T, H, dk, dv, int(chunk), dt, _ptr(o), _ptr(hT),
                             _ptr(workspace), ws_bytes, _stream(stream))
    _raise_on(st, "gla_chunk_fwd")
    return o, hT


def gla_chunk_fwd_noalloc(q, k, v, log_lambda, h0=None, scale=None, chunk=128, *, o, hT=None, stream=None):
    """The forward without any device allocation by the library: for callers
    that may not allocate device memory, the segmentation scratch comes from
    a fixed array inside the library. The caller passes the output tensors.
    Returns (o, hT)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    st = lib().gla_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), float(scale),
                                     B, T, H, dk, dv, int(chunk), _dtype_code(q), _ptr(o), _ptr(hT),
                                     _stream(stream))
    _raise_on(st, "gla_chunk_fwd_noalloc")
    return o, hT


def gla_chunk_fwd_varlen(q, k, v, log_lambda, cu_seqlens, state_pool, slots=None, scale=None, chunk=128, *,
                         o=None, stream=None):
    """Variable-length forward: q, k [total_T,H,dk], v [total_T,H,dv] bf16
    packed, sequence n = tokens [cu_seqlens[n], cu_seqlens[n+1]) (int32 CUDA
    tensor), state_pool [n_slots,H,dk,dv] fp32 updated in place at slots[n]
    (int32 CUDA tensor, or None for slot n). Returns o [total_T,H,dv]."""
    torch = _torch()
    total_T, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if o is None:
        o = torch.empty((total_T, H, dv), dtype=q.dtype, device=q.device)
    nseq = cu_seqlens.numel() - 1
    st = lib().gla_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), float(scale), _ptr(cu_seqlens),
                                    _ptr(slots), _ptr(state_pool), int(state_pool.shape[0]), nseq, total_T, H,
                                    dk, dv, int(chunk), _dtype_code(q), _ptr(o), _stream(stream))
    _raise_on(st, "gla_chunk_fwd_varlen")
    return o


def gla_chunk_fwd_gated_workspace_size(B, T, H, dk, dv, chunk=128, dtype=GLA_BF16) -> int:
    return int(lib().gla_chunk_fwd_gated_workspace_size(B, T, H, dk, dv, chunk, dtype))


def gla_chunk_fwd_gated(q, k, v, g, h0=None, scale=None, chunk=128, *, o=None, hT=None, want_hT=True,
                        workspace=None, stream=None):
    """Chunked forward with a per-token decay: g [B,T,H] fp32 natural-log
    decays (<= 0, -inf clears the state); q, k, v, h0 as gla_chunk_fwd.
    Returns (o, hT)."""
    torch = _torch()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if hT is None and want_hT:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    dt = _dtype_code(q)
    ws_need = gla_chunk_fwd_gated_workspace_size(B, T, H, dk, dv, chunk, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gla_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _f32(g, (B, T, H), "g"), _f32(h0, (B, H, dk, dv), "h0"),
                                   float(scale), B, T, H, dk, dv,
                                   int(chunk), dt, _ptr(o), _ptr(hT), _ptr(workspace), ws_bytes, _stream(stream))
    _raise_on(st, "gla_chunk_fwd_gated")
    return o, hT


def gla_chunk_fwd_varlen_gated(q, k, v, g, cu_seqlens, state_pool, slots=None, scale=None, chunk=128, *,
                               o=None, stream=None):
    """Variable-length forward with a per-token decay: g [total_T,H] fp32
    natural-log decays, packed like q; otherwise as gla_chunk_fwd_varlen.
    Returns o [total_T,H,dv]."""
    torch = _torch()
    total_T, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if o is None:
        o = torch.empty((total_T, H, dv), dtype=q.dtype, device=q.device)
    nseq = cu_seqlens.numel() - 1
    st = lib().gla_chunk_fwd_varlen_gated(_ptr(q), _ptr(k), _ptr(v), _f32(g, (total_T, H), "g"), float(scale),
                                          _ptr(cu_seqlens),
                                          _ptr(slots), _ptr(state_pool), int(state_pool.shape[0]), nseq, total_T, H,
                                          dk, dv, int(chunk), _dtype_code(q), _ptr(o), _stream(stream))
    _raise_on(st, "gla_chunk_fwd_varlen_gated")
    return o


def gla_chunk_fwd_mixer(q, k, v, g, log_lambda, h0=None, scale=None, chunk=128, aug=None, norm_w=None, eps=1e-6,
                        *, z=None, hT=None, want_hT=True, workspace=None, stream=None):
    """The chunked forward followed by the mixer epilogue, z in place of o
    (bf16): returns (z, hT), z [B,T,H,dv] = Head RMSNorm(o + sigmoid(q.(aug*k)) v)
    * norm_w * SiLU(g)."""
    torch = _torch()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if z is None:
        z = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if hT is None and want_hT:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = gla_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device) if n else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gla_chunk_fwd_mixer(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(log_lambda), _ptr(h0), float(scale),
                                   _ptr(aug), _ptr(norm_w), float(eps), B, T, H, dk, dv, int(chunk), _dtype_code(q),
                                   _ptr(z), _ptr(hT), _ptr(workspace), ws_bytes, _stream(stream))
    _raise_on(st, "gla_chunk_fwd_mixer")
    return z, hT


def gla_chunk_bwd(q, k, v, log_lambda, do, h0=None, dhT=None, scale=None, chunk=128, *,
                  dq=None, dk=None, dv=None, dh0=None, want_dh0=True, workspace=None, stream=None):
    """Chunked backward. Returns (dq, dk, dv, dh0)."""
    torch = _torch()
    B, T, H, dk_ = q.shape
    dv_ = v.shape[-1]
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(dk_)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dh0 is None and want_dh0:
        dh0 = torch.empty((B, H, dk_, dv_), dtype=torch.float32, device=q.device)
    ws_need = gla_chunk_bwd_workspace_size(B, T, H, dk_, dv_, chunk, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gla_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), float(scale),
                             _ptr(do), _ptr(dhT), B, T, H, dk_, dv_, int(chunk), dt,
                             _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dh0), _ptr(workspace), ws_bytes,
                             _stream(stream))
    _raise_on(st, "gla_chunk_bwd")
    return dq, dk, dv, dh0


def gla_chunk_bwd_gated_workspace_size(B, T, H, dk, dv, chunk=128, dtype=GLA_BF16) -> int:
    return int(lib().gla_chunk_bwd_gated_workspace_size(B, T, H, dk, dv, chunk, dtype))


def gla_chunk_bwd_gated(q, k, v, g, do, h0=None, dhT=None, scale=None, chunk=128, *,
                        dq=None, dk=None, dv=None, dh0=None, dg=None, want_dh0=True, workspace=None, stream=None):
    """Chunked backward with a per-token decay: g [B,T,H] fp32 natural-log
    decays as gla_chunk_fwd_gated; otherwise as gla_chunk_bwd. Returns
    (dq, dk, dv, dh0, dg), dg [B,T,H] fp32."""
    torch = _torch()
    B, T, H, dk_ = q.shape
    dv_ = v.shape[-1]
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(dk_)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dh0 is None and want_dh0:
        dh0 = torch.empty((B, H, dk_, dv_), dtype=torch.float32, device=q.device)
    if dg is None:
        dg = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    ws_need = gla_chunk_bwd_gated_workspace_size(B, T, H, dk_, dv_, chunk, dt)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gla_chunk_bwd_gated(_ptr(q), _ptr(k), _ptr(v), _f32(g, (B, T, H), "g"),
                                   _f32(h0, (B, H, dk_, dv_), "h0"), float(scale), _ptr(do),
                                   _f32(dhT, (B, H, dk_, dv_), "dhT"), B, T, H, dk_, dv_, int(chunk), dt,
                                   _ptr(dq), _ptr(dk), _ptr(dv), _f32(dh0, (B, H, dk_, dv_), "dh0"),
                                   _f32(dg, (B, T, H), "dg"), _ptr(workspace), ws_bytes, _stream(stream))
    _raise_on(st, "gla_chunk_bwd_gated")
    return dq, dk, dv, dh0, dg


def gla_decode_step(q, k, v, log_lambda, S, scale=None, *, o=None, stream=None):
    """One recurrent step. q, k [N,H,dk], v [N,H,dv], S [N,H,dk,dv] fp32
    (updated in place). Returns o [N,H,dv]."""
    torch = _torch()
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    st = lib().gla_decode_step(_ptr(q), _ptr(k), _ptr(v), _f32(log_lambda, (H,), "log_lambda"),
                               _f32(S, (N, H, dk, dv), "S"), float(scale),
                               N, H, dk, dv, dt, _ptr(o), _stream(stream))
    _raise_on(st, "gla_decode_step")
    return o


def gla_decode_step_gated(q, k, v, g, S, scale=None, *, o=None, stream=None):
    """One recurrent step with a per-token decay g [N,H] fp32 (natural log).
    S [N,H,dk,dv] fp32 is updated in place. Returns o [N,H,dv]."""
    torch = _torch()
    N, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    st = lib().gla_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _f32(g, (N, H), "g"), _f32(S, (N, H, dk, dv), "S"),
                                     float(scale), N, H, dk, dv,
                                     _dtype_code(q), _ptr(o), _stream(stream))
    _raise_on(st, "gla_decode_step_gated")
    return o


def gla_decode_step_mixer(q, k, v, log_lambda, S, g, aug=None, norm_w=None, eps=1e-6, scale=None, *, z=None,
                          stream=None):
    """Decode step plus the mixer epilogue in one kernel. Returns z [N,H,dv]."""
    torch = _torch()
    N, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if z is None:
        z = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    st = lib().gla_decode_step_mixer(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(S), float(scale), _ptr(g),
                                     _ptr(aug), _ptr(norm_w), float(eps), N, H, dk, dv, _dtype_code(q), _ptr(z),
                                     _stream(stream))
    _raise_on(st, "gla_decode_step_mixer")
    return z


def gla_mixer_epilogue(o, q, k, v, g, aug=None, norm_w=None, eps=1e-6, *, z=None, stream=None):
    """The mixer epilogue over [..., H, d] rows (any leading dims). Returns z like o."""
    torch = _torch()
    H, dv = o.shape[-2], o.shape[-1]
    dk = q.shape[-1]
    NT = o.numel() // (H * dv)
    if z is None:
        z = torch.empty_like(o)
    st = lib().gla_mixer_epilogue(_ptr(o), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(aug), _ptr(norm_w), float(eps),
                                  NT, H, dk, dv, _dtype_code(o), _ptr(z), _stream(stream))
    _raise_on(st, "gla_mixer_epilogue")
    return z


def gla_conv1d_fwd(x, w, b=None, win_in=None, *, y=None, win_out=None, want_window=True, stream=None):
    """Causal depthwise Conv1d (width 4) + SiLU over x [B,T,D]; w [D,4], b [D]
    fp32; win_in [B,4,D] fp32 or None (zeros). Returns (y, win_out); win_out
    may be win_in (in place), or None with want_window=False."""
    torch = _torch()
    B, T, D = x.shape
    if y is None:
        y = torch.empty_like(x)
    if win_out is None and want_window:
        win_out = torch.empty((B, 4, D), dtype=torch.float32, device=x.device)
    st = lib().gla_conv1d_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(win_in), B, T, D, _dtype_code(x), _ptr(y),
                              _ptr(win_out), _stream(stream))
    _raise_on(st, "gla_conv1d_fwd")
    return y, win_out


def gla_conv1d_varlen(x, w, b, cu_seqlens, win_pool, slots=None, *, y=None, stream=None):
    """The Conv1d over packed sequences x [total_T,D] (cu_seqlens int32 CUDA
    tensor), windows in win_pool [n_slots,4,D] fp32 at slots[n] (int32 CUDA
    tensor, or None for slot n), updated in place. Returns y [total_T,D]."""
    torch = _torch()
    total_T, D = x.shape
    if y is None:
        y = torch.empty_like(x)
    nseq = cu_seqlens.numel() - 1
    st = lib().gla_conv1d_varlen(_ptr(x), _ptr(w), _ptr(b), _ptr(cu_seqlens), _ptr(slots), _ptr(win_pool),
                                 int(win_pool.shape[0]), nseq, total_T, D, _dtype_code(x), _ptr(y), _stream(stream))
    _raise_on(st, "gla_conv1d_varlen")
    return y


def gla_conv1d_step(x, w, b, win, *, y=None, stream=None):
    """One serving step of the Conv1d: x [N,D], win [N,4,D] fp32 updated in
    place. Returns y [N,D]."""
    torch = _torch()
    N, D = x.shape
    if y is None:
        y = torch.empty_like(x)
    st = lib().gla_conv1d_step(_ptr(x), _ptr(w), _ptr(b), _ptr(win), N, D, _dtype_code(x), _ptr(y), _stream(stream))
    _raise_on(st, "gla_conv1d_step")
    return y


class _Call:
    """The tensors of one call: all on the device of the first, each checked
    for type and shape before its address is taken. The call runs with that
    device current, on `stream` or the device's current stream; what it
    allocates (outputs, workspace) belongs to the stream it runs on. Kept
    lean: a serving step's kernels take a few microseconds."""

    __slots__ = ("torch", "device", "index", "here", "dtype", "code", "stream", "other", "kept", "f")

    def __init__(self, x, stream, element=True):
        self.torch = torch = _torch()
        self.device = x.device
        self.index = x.get_device()
        if self.index < 0:
            raise GlaError(GLA_ERR_INVALID_ARG, "argument", "tensors must live on a CUDA device")
        self.here = self.index == torch.cuda.current_device()
        self.dtype = x.dtype
        self.code = _dtype_code(x) if element else None
        self.f = torch.float32
        self.other = None
        current = torch._C._cuda_getCurrentRawStream(self.index)
        self.stream = current if stream is None else _stream(stream)
        if self.stream != current:
            cuda = torch.cuda
            if hasattr(stream, "cuda_stream"):
                self.other = stream
            else:
                self.other = cuda.ExternalStream(self.stream, self.device) if self.stream else cuda.default_stream(self.device)

    def _refuse(self, t, shape, dtype, name):
        if t.get_device() != self.index:
            raise GlaError(GLA_ERR_INVALID_ARG, "argument",
                           f"{name} is on {t.device}, the call's tensors on {self.device}")
        if t.dtype != dtype:
            raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")

    def whole(self, t, shape, name, dtype=None):
        """Address of a contiguous tensor (None passes); dtype None: the call's element type."""
        if t is None:
            return None
        if dtype is None:
            dtype = self.dtype
        if t.dtype is dtype and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t.data_ptr()
        self._refuse(t, shape, dtype, name)
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} must be contiguous")

    def f32(self, t, shape, name):
        if t is None:
            return None
        if t.dtype is self.f and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t.data_ptr()
        return self.whole(t, shape, name, self.f)

    def i32(self, t, shape, name):
        return self.whole(t, shape, name, self.torch.int32)

    def rows(self, t, shape, name):
        """Address and row step of [..., C] rows an equal distance apart with
        contiguous columns (a column range of a wider tensor passes)."""
        if t is None:
            return None, 0
        if t.dtype is self.dtype and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t.data_ptr(), shape[-1]
        self._refuse(t, shape, self.dtype, name)
        if t.numel() == 0:
            return t.data_ptr(), shape[-1]
        lead = [(n, st) for n, st in zip(shape[:-1], t.stride()[:-1]) if n > 1]
        step = lead[-1][1] if lead else shape[-1]
        if t.stride(-1) != 1 and shape[-1] > 1 or len(lead) == 2 and lead[0][1] != lead[1][0] * step or step < shape[-1]:
            raise GlaError(GLA_ERR_INVALID_ARG, "argument",
                           f"{name} must have contiguous columns and token rows an equal distance apart")
        return t.data_ptr(), step

    def empty(self, shape, dtype=None):
        """A new tensor on the call's device and stream."""
        dtype = self.dtype if dtype is None else dtype
        if self.other is None:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        with self.torch.cuda.stream(self.other):
            return self.torch.empty(shape, dtype=dtype, device=self.device)

    def scratch(self, workspace, size, *shape):
        """Address and bytes of the caller's workspace, or of a new one of
        size(*shape) bytes, asked with the call's device current: the plan
        behind it depends on that device's SMs. size None: no workspace."""
        if workspace is None:
            if size is None:
                return None, 0
            if self.here:
                need = size(*shape, self.code)
            else:
                with self.torch.cuda.device(self.index):
                    need = size(*shape, self.code)
            if need == 0:
                return None, 0
            self.kept = self.empty(need, self.torch.uint8)
            return self.kept.data_ptr(), need
        if workspace.get_device() != self.index or not workspace.is_contiguous():
            raise GlaError(GLA_ERR_INVALID_ARG, "argument", "the workspace must be contiguous and on the call's device")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()

    def run(self, name, *args):
        f = _entry.get(name)
        if f is None:
            f = _entry[name] = getattr(lib(), name)
        if self.here:
            st = f(*args, self.stream)
        else:
            with self.torch.cuda.device(self.index):
                st = f(*args, self.stream)
        if st != GLA_OK:
            _raise_on(st, name)


_entry = {}   # entry points already looked up


def _lead(t, n, name):
    shape = t.shape
    if len(shape) != n:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} has {len(shape)} dimensions, expected {n}")
    return shape


def _ssm_rows(c, x, dt, A, Bm, Cm, skip, z, dt_bias, softplus):
    """The arguments every selective-scan entry point begins with."""
    wide = x.shape
    D, N = wide[-1], _lead(A, 2, "A")[1]
    narrow = wide[:-1] + (N,)
    return (*c.rows(x, wide, "x"), *c.rows(dt, wide, "dt"), c.f32(A, (D, N), "A"), *c.rows(Bm, narrow, "Bm"),
            *c.rows(Cm, narrow, "Cm"), c.f32(skip, (D,), "skip"), *c.rows(z, wide, "z"),
            c.f32(dt_bias, (D,), "dt_bias"), 1 if softplus else 0)


def gla_ssm_fwd_workspace_size(B, T, D, N, dtype=GLA_BF16) -> int:
    return int(lib().gla_ssm_fwd_workspace_size(B, T, D, N, dtype))


def gla_ssm_varlen_workspace_size(nseq, total_T, D, N, dtype=GLA_BF16) -> int:
    return int(lib().gla_ssm_varlen_workspace_size(nseq, total_T, D, N, dtype))


def gla_ssm_fwd(x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, h0=None, *, softplus=True, y=None, hT=None,
                want_hT=True, workspace=None, stream=None):
    """The selective state-space scan: x, dt, z [B,T,D], Bm, Cm [B,T,N] (bf16
    or fp32; column ranges of wider tensors pass), A [D,N], skip, dt_bias [D]
    fp32, h0 [B,D,N] fp32 or None (zeros). With delta = softplus(dt + dt_bias),
    h = exp(delta A) h + delta B x, y = (C.h + skip x) SiLU(z). Returns
    (y [B,T,D], hT [B,D,N] fp32; hT may be h0)."""
    B, T, D = _lead(x, 3, "x")
    c = _Call(x, stream)
    args = _ssm_rows(c, x, dt, A, Bm, Cm, skip, z, dt_bias, softplus)
    N = A.shape[1]
    if y is None:
        y = c.empty((B, T, D))
    if hT is None and want_hT:
        hT = c.empty((B, D, N), c.torch.float32)
    c.run("gla_ssm_fwd", *args, c.f32(h0, (B, D, N), "h0"), B, T, D, N, c.code, c.whole(y, (B, T, D), "y"),
          c.f32(hT, (B, D, N), "hT"), *c.scratch(workspace, gla_ssm_fwd_workspace_size, B, T, D, N))
    return y, hT


def _pools(c, n, D, N, state_pool, slots, conv_w, conv_b, win_pool):
    k = _lead(state_pool, 3, "state_pool")[0]
    return (c.f32(conv_w, (D, 4), "conv_w"), c.f32(conv_b, (D,), "conv_b"), c.i32(slots, (n,), "slots"),
            c.f32(state_pool, (k, D, N), "state_pool"), c.f32(win_pool, (k, 4, D), "win_pool"), k)


def gla_ssm_varlen(x, dt, A, Bm, Cm, cu_seqlens, state_pool, skip=None, z=None, dt_bias=None, slots=None, *,
                   conv_w=None, conv_b=None, win_pool=None, softplus=True, y=None, workspace=None, stream=None):
    """The selective scan over packed sequences: x, dt, z [total_T,D], Bm, Cm
    [total_T,N], sequence n = tokens [cu_seqlens[n], cu_seqlens[n+1]) (int32
    CUDA tensor), state_pool [n_slots,D,N] fp32 updated in place at slots[n]
    (int32 CUDA tensor, or None for slot n). With conv_w [D,4] (and conv_b [D],
    win_pool [n_slots,4,D], fp32) x goes through the causal Conv1d with SiLU
    first, its windows updated in place. Returns y [total_T,D]."""
    total_T, D = _lead(x, 2, "x")
    c = _Call(x, stream)
    args = _ssm_rows(c, x, dt, A, Bm, Cm, skip, z, dt_bias, softplus)
    N, nseq = A.shape[1], cu_seqlens.numel() - 1
    w, b, sl, pool, win, k = _pools(c, nseq, D, N, state_pool, slots, conv_w, conv_b, win_pool)
    if y is None:
        y = c.empty((total_T, D))
    c.run("gla_ssm_varlen", *args, w, b, c.i32(cu_seqlens, (nseq + 1,), "cu_seqlens"), sl, pool, win, k, nseq,
          total_T, D, N, c.code, c.whole(y, (total_T, D), "y"),
          *c.scratch(workspace, gla_ssm_varlen_workspace_size, nseq, total_T, D, N))
    return y


def gla_ssm_step(x, dt, A, Bm, Cm, state_pool, skip=None, z=None, dt_bias=None, slots=None, *, conv_w=None,
                 conv_b=None, win_pool=None, softplus=True, y=None, stream=None):
    """One token per sequence of the selective scan: x, dt, z [N,D], Bm, Cm
    [N,n]; pools, slots and the Conv1d as gla_ssm_varlen. Returns y [N,D]."""
    n, D = _lead(x, 2, "x")
    c = _Call(x, stream)
    args = _ssm_rows(c, x, dt, A, Bm, Cm, skip, z, dt_bias, softplus)
    N = A.shape[1]
    w, b, sl, pool, win, k = _pools(c, n, D, N, state_pool, slots, conv_w, conv_b, win_pool)
    if y is None:
        y = c.empty((n, D))
    c.run("gla_ssm_step", *args, w, b, sl, pool, win, k, n, D, N, c.code, c.whole(y, (n, D), "y"))
    return y


def gla_ssm_bwd_workspace_size(B, T, D, N, dtype=GLA_BF16) -> int:
    return int(lib().gla_ssm_bwd_workspace_size(B, T, D, N, dtype))


def gla_ssm_bwd(x, dt, A, Bm, Cm, dy, skip=None, z=None, dt_bias=None, h0=None, dhT=None, *, softplus=True, dx=None,
                ddt=None, dA=None, dB=None, dC=None, dskip=None, dz=None, ddt_bias=None, dh0=None, want_dh0=True,
                workspace=None, stream=None):
    """Gradients of gla_ssm_fwd (the same inputs; dy [B,T,D] for y, dhT
    [B,D,N] fp32 or None for hT). Returns (dx, ddt, dA, dB, dC, dskip, dz,
    ddt_bias, dh0): dskip, dz and ddt_bias are None where skip, z and dt_bias
    are, dh0 with want_dh0=False."""
    B, T, D = _lead(x, 3, "x")
    c = _Call(x, stream)
    args = _ssm_rows(c, x, dt, A, Bm, Cm, skip, z, dt_bias, softplus)
    N = A.shape[1]
    f32, wide, narrow, state = c.torch.float32, (B, T, D), (B, T, N), (B, D, N)
    args += (c.f32(h0, state, "h0"), *c.rows(dy, wide, "dy"), c.f32(dhT, state, "dhT"), B, T, D, N, c.code)
    dx = c.empty(wide) if dx is None else dx
    ddt = c.empty(wide) if ddt is None else ddt
    dA = c.empty((D, N), f32) if dA is None else dA
    dB = c.empty(narrow) if dB is None else dB
    dC = c.empty(narrow) if dC is None else dC
    if dskip is None and skip is not None:
        dskip = c.empty((D,), f32)
    if dz is None and z is not None:
        dz = c.empty(wide)
    if ddt_bias is None and dt_bias is not None:
        ddt_bias = c.empty((D,), f32)
    if dh0 is None and want_dh0:
        dh0 = c.empty(state, f32)
    c.run("gla_ssm_bwd", *args, c.whole(dx, wide, "dx"), c.whole(ddt, wide, "ddt"), c.f32(dA, (D, N), "dA"),
          c.whole(dB, narrow, "dB"), c.whole(dC, narrow, "dC"), c.f32(dskip, (D,), "dskip"), c.whole(dz, wide, "dz"),
          c.f32(ddt_bias, (D,), "ddt_bias"), c.f32(dh0, state, "dh0"),
          *c.scratch(workspace, gla_ssm_bwd_workspace_size, B, T, D, N))
    return dx, ddt, dA, dB, dC, dskip, dz, ddt_bias, dh0


def gla_conv1d_bwd_workspace_size(B, T, D, dtype=GLA_BF16) -> int:
    return int(lib().gla_conv1d_bwd_workspace_size(B, T, D, dtype))


def gla_conv1d_bwd(x, w, b, dy, win_in=None, *, dx=None, dw=None, db=None, want_db=True, workspace=None, stream=None):
    """Gradients of gla_conv1d_fwd (its y without the window it leaves): x, dy
    [B,T,D], w [D,4], b [D] or None, win_in [B,4,D] or None (a constant).
    Returns (dx, dw, db); db None with want_db=False."""
    B, T, D = _lead(x, 3, "x")
    c = _Call(x, stream)
    f32 = c.torch.float32
    args = (c.whole(x, x.shape, "x"), c.f32(w, (D, 4), "w"), c.f32(b, (D,), "b"), c.whole(dy, x.shape, "dy"),
            c.f32(win_in, (B, 4, D), "win_in"))
    dx = c.empty((B, T, D)) if dx is None else dx
    dw = c.empty((D, 4), f32) if dw is None else dw
    if db is None and want_db:
        db = c.empty((D,), f32)
    c.run("gla_conv1d_bwd", *args, B, T, D, c.code, c.whole(dx, x.shape, "dx"), c.f32(dw, (D, 4), "dw"),
          c.f32(db, (D,), "db"), *c.scratch(workspace, gla_conv1d_bwd_workspace_size, B, T, D))
    return dx, dw, db


def _norm_rows(x):
    if x.dim() < 1:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", "x has no channels")
    D = x.shape[-1]
    return (x.numel() // D if D else 0), D


def gla_rmsnorm(x, w=None, res=None, eps=1e-6, *, y=None, s=None, stream=None):
    """Residual addition and RMSNorm over the last dimension: x, res [..., D],
    w [D] fp32 or None. Returns (y, s): s = x + res (may be given as res, in
    place), or None without res; y = s w / sqrt(mean(s^2) + eps)."""
    rows, D = _norm_rows(x)
    c = _Call(x, stream)
    y = c.empty(x.shape) if y is None else y
    if s is None and res is not None:
        s = c.empty(x.shape)
    c.run("gla_rmsnorm_fwd", c.whole(x, x.shape, "x"), c.whole(res, x.shape, "res"), c.f32(w, (D,), "w"), float(eps),
          rows, D, 0, c.code, c.whole(s, x.shape, "s"), c.whole(y, x.shape, "y"), None, None)
    return y, s


def gla_rmsnorm_q8(x, w=None, res=None, eps=1e-6, group=128, *, y8=None, scale=None, s=None, stream=None):
    """gla_rmsnorm with its output in 8 bits: y8 [..., D] float8_e4m3fn and
    scale fp32, y = y8 * scale: [..., ceil(D / group)] for group 32, 64 or 128
    channels a scale, [..., 1] for group 0 (one a row). Returns (y8, scale, s)."""
    rows, D = _norm_rows(x)
    c = _Call(x, stream)
    shape = x.shape[:-1] + (-(-D // group) if group > 0 else 1,)
    y8 = c.empty(x.shape, c.torch.float8_e4m3fn) if y8 is None else y8
    scale = c.empty(shape, c.torch.float32) if scale is None else scale
    if s is None and res is not None:
        s = c.empty(x.shape)
    c.run("gla_rmsnorm_fwd", c.whole(x, x.shape, "x"), c.whole(res, x.shape, "res"), c.f32(w, (D,), "w"), float(eps),
          rows, D, int(group), c.code, c.whole(s, x.shape, "s"), None,
          c.whole(y8, x.shape, "y8", c.torch.float8_e4m3fn), c.f32(scale, shape, "scale"))
    return y8, scale, s


def gla_rmsnorm_bwd_workspace_size(rows, D, dtype=GLA_BF16) -> int:
    return int(lib().gla_rmsnorm_bwd_workspace_size(rows, D, dtype))


def gla_rmsnorm_bwd(s, w, dy, ds=None, eps=1e-6, *, dx=None, dw=None, want_dw=True, workspace=None, stream=None):
    """Gradients of gla_rmsnorm: s (x + res, or x), dy, ds (the gradient that
    reaches s itself, or None) [..., D], w [D] or None. Returns (dx, dw): dx is
    x's and res's alike, dw [D] fp32 (None with want_dw=False)."""
    rows, D = _norm_rows(s)
    c = _Call(s, stream)
    args = (c.whole(s, s.shape, "s"), c.f32(w, (D,), "w"), c.whole(dy, s.shape, "dy"), c.whole(ds, s.shape, "ds"))
    dx = c.empty(s.shape) if dx is None else dx
    if dw is None and want_dw:
        dw = c.empty((D,), c.torch.float32)
    size = None if dw is None else gla_rmsnorm_bwd_workspace_size
    c.run("gla_rmsnorm_bwd", *args, float(eps), rows, D, c.code, c.whole(dx, s.shape, "dx"), c.f32(dw, (D,), "dw"),
          *c.scratch(workspace, size, rows, D))
    return dx, dw


class _Quick:
    """One call's device and stream, for operators whose small calls cost the
    host more than the GPU: on the current device and its current stream next
    to nothing is set up, for any other a _Call does the work."""

    __slots__ = ("torch", "index", "device", "call")

    def __init__(self, x, stream, element=True):
        torch = self.torch = _torch()
        index = self.index = x.get_device()
        self.device = x.device
        here = stream is None and index >= 0 and index == torch._C._cuda_getDevice()
        self.call = None if here else _Call(x, stream, element)

    def empty(self, shape, dtype):
        if self.call is None:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        return self.call.empty(shape, dtype)

    def run(self, name, *args):
        if self.call is not None:
            return self.call.run(name, *args)
        f = _entry.get(name)
        if f is None:
            f = _entry[name] = getattr(lib(), name)
        st = f(*args, self.torch._C._cuda_getCurrentRawStream(self.index))
        if st != GLA_OK:
            _raise_on(st, name)


def _at(t, dtype, shape, index, name):
    """Address of a contiguous tensor of this type, shape and device (None passes)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != index:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} is on {t.device}, not on the call's device {index}")
    if t.dtype != dtype:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise GlaError(GLA_ERR_INVALID_ARG, "argument", f"{name} must be contiguous")


def gla_layernorm(x, w=None, b=None, res=None, eps=1e-6, *, y=None, s=None, stream=None):
    """Residual addition and layer norm over the last dimension: x, res [..., D],
    w, b [D] fp32 or None. Returns (y, s): s = x + res (may be given as res, in
    place), or None without res; y = w (s - mean(s)) / sqrt(var(s) + eps) + b."""
    rows, D = _norm_rows(x)
    c = _Quick(x, stream)
    index, dtype, shape, f32 = c.index, x.dtype, x.shape, c.torch.float32
    if y is None:
        y = c.empty(shape, dtype)
    if s is None and res is not None:
        s = c.empty(shape, dtype)
    c.run("gla_layernorm_fwd", _at(x, dtype, shape, index, "x"), _at(res, dtype, shape, index, "res"),
          _at(w, f32, (D,), index, "w"), _at(b, f32, (D,), index, "b"), eps, rows, D, _dtype_code(x),
          _at(s, dtype, shape, index, "s"), _at(y, dtype, shape, index, "y"))
    return y, s


def gla_layernorm_bwd_workspace_size(rows, D, dtype=GLA_BF16) -> int:
    return int(lib().gla_layernorm_bwd_workspace_size(rows, D, dtype))


def gla_layernorm_bwd(s, w, dy, ds=None, eps=1e-6, *, dx=None, dw=None, db=None, want_dw=True, want_db=True,
                      workspace=None, stream=None):
    """Gradients of gla_layernorm: s (x + res, or x), dy, ds (the gradient that
    reaches s itself, or None) [..., D], w [D] or None. Returns (dx, dw, db):
    dx is x's and res's alike, dw and db [D] fp32 (None with want_dw=False,
    want_db=False)."""
    rows, D = _norm_rows(s)
    c = _Quick(s, stream)
    index, dtype, shape, f32, code = c.index, s.dtype, s.shape, c.torch.float32, _dtype_code(s)
    args = (_at(s, dtype, shape, index, "s"), _at(w, f32, (D,), index, "w"), _at(dy, dtype, shape, index, "dy"),
            _at(ds, dtype, shape, index, "ds"))
    if dx is None:
        dx = c.empty(shape, dtype)
    if dw is None and want_dw:
        dw = c.empty((D,), f32)
    if db is None and want_db:
        db = c.empty((D,), f32)
    size = None if dw is None and db is None else gla_layernorm_bwd_workspace_size
    if c.call is None and workspace is None and size is not None:
        need = size(rows, D, code)
        workspace = c.empty((need,), c.torch.uint8)
        scratch = workspace.data_ptr(), need
    else:
        scratch = (c.call or _Call(s, None)).scratch(workspace, size, rows, D)
    c.run("gla_layernorm_bwd", *args, eps, rows, D, code, _at(dx, dtype, shape, index, "dx"),
          _at(dw, f32, (D,), index, "dw"), _at(db, f32, (D,), index, "db"), *scratch)
    return dx, dw, db


def _heads(t, dtype, shape, index, name):
    """Address and row step of [T, H, d] token rows an equal distance apart,
    each with contiguous heads (a column range of a wider tensor passes)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        T, H, d = shape
        if t.is_contiguous():
            return t.data_ptr(), H * d
        step = t.stride(0) if T > 1 else H * d
        if not (d > 1 and t.stride(2) != 1 or H > 1 and t.stride(1) != d or step < H * d):
            return t.data_ptr(), step
        raise GlaError(GLA_ERR_INVALID_ARG, "argument",
                       f"{name} must have contiguous heads and token rows an equal distance apart")
    return _at(t, dtype, shape, index, name), shape[1] * shape[2]


def _rows(t, dtype, shape, index, name):
    """Address and row step of [T, D] rows an equal distance apart with contiguous columns (None passes)."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        T, D = shape
        if t.is_contiguous():
            return t.data_ptr(), D
        step = t.stride(0) if T > 1 else D
        if not (D > 1 and t.stride(1) != 1 or step < D):
            return t.data_ptr(), step
        raise GlaError(GLA_ERR_INVALID_ARG, "argument",
                       f"{name} must have contiguous columns and token rows an equal distance apart")
    return _at(t, dtype, shape, index, name), shape[1]


def _offsets(cu_nodes):
    shape = cu_nodes.shape
    if len(shape) != 1 or shape[0] < 1:
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", "cu_nodes must hold one offset more than there are sequences")
    return shape


def _tree_fwd(name, q, k, v, decay, gated, cu_nodes, parents, state_pool, slots, scale, o, stream):
    T, H, dk = _lead(q, 3, "q")
    dv = _lead(v, 3, "v")[2]
    c = _Quick(q, stream)
    index, dtype, i32, f32, cu = c.index, q.dtype, c.torch.int32, c.torch.float32, _offsets(cu_nodes)
    narrow, wide, nseq, n_slots = (T, H, dk), (T, H, dv), cu[0] - 1, _lead(state_pool, 4, "state_pool")[0]
    args = (*_heads(q, dtype, narrow, index, "q"), *_heads(k, dtype, narrow, index, "k"),
            *_heads(v, dtype, wide, index, "v"), _at(decay, f32, (T, H) if gated else (H,), index, "g" if gated else "log_lambda"),
            (dk or 1) ** -0.5 if scale is None else scale, _at(cu_nodes, i32, cu, index, "cu_nodes"),
            _at(parents, i32, (T,), index, "parents"), _at(slots, i32, (nseq,), index, "slots"),
            _at(state_pool, f32, (n_slots, H, dk, dv), index, "state_pool"), n_slots, nseq, T, H, dk, dv, _dtype_code(q))
    if o is None:
        o = c.empty(wide, dtype)
    c.run(name, *args, _at(o, dtype, wide, index, "o"))
    return o


def gla_tree_fwd(q, k, v, log_lambda, cu_nodes, parents, state_pool, slots=None, scale=None, *, o=None, stream=None):
    """The outputs of drafted tokens: trees packed one behind another, tree n =
    nodes [cu_nodes[n], cu_nodes[n+1]) (int32 CUDA tensor, at most 64 each),
    parents [T] int32 (within the tree, before the node; -1: the sequence's
    state). q, k [T,H,dk], v [T,H,dv] (column ranges of wider tensors pass),
    state_pool [n_slots,H,dk,dv] fp32, read at slots[n] (int32 CUDA tensor, or
    None for slot n) and left as it is. Returns o [T,H,dv]: what
    gla_decode_step would give along each node's path (at bf16 with the page's
    entries and the decayed scores as two bf16 each, 2^-17 of themselves, before
    the one rounding of o; fp32 throughout at fp32)."""
    return _tree_fwd("gla_tree_fwd", q, k, v, log_lambda, False, cu_nodes, parents, state_pool, slots, scale, o, stream)


def gla_tree_fwd_gated(q, k, v, g, cu_nodes, parents, state_pool, slots=None, scale=None, *, o=None, stream=None):
    """gla_tree_fwd with a decay per node: g [T,H] fp32 (natural log, <= 0;
    -inf clears the state along the node's path)."""
    return _tree_fwd("gla_tree_fwd_gated", q, k, v, g, True, cu_nodes, parents, state_pool, slots, scale, o, stream)


def _tree_commit(name, k, v, decay, gated, cu_nodes, parents, last, state_pool, slots, x, win_pool, stream):
    T, H, dk = _lead(k, 3, "k")
    dv = _lead(v, 3, "v")[2]
    c = _Quick(k, stream)
    index, dtype, i32, f32, cu = c.index, k.dtype, c.torch.int32, c.torch.float32, _offsets(cu_nodes)
    nseq, n_slots, D = cu[0] - 1, _lead(state_pool, 4, "state_pool")[0], 0 if x is None else _lead(x, 2, "x")[1]
    c.run(name, *_heads(k, dtype, (T, H, dk), index, "k"), *_heads(v, dtype, (T, H, dv), index, "v"),
          _at(decay, f32, (T, H) if gated else (H,), index, "g" if gated else "log_lambda"),
          _at(cu_nodes, i32, cu, index, "cu_nodes"), _at(parents, i32, (T,), index, "parents"),
          _at(last, i32, (nseq,), index, "last"), _at(slots, i32, (nseq,), index, "slots"),
          _at(state_pool, f32, (n_slots, H, dk, dv), index, "state_pool"), *_rows(x, dtype, (T, D), index, "x"),
          _at(win_pool, f32, (n_slots, 4, D), index, "win_pool"), n_slots, nseq, T, H, dk, dv, D, _dtype_code(k))
    return state_pool


def gla_tree_commit(k, v, log_lambda, cu_nodes, parents, last, state_pool, slots=None, *, x=None, win_pool=None,
                    stream=None):
    """Keeps the accepted path of each tree of gla_tree_fwd: state_pool
    [n_slots,H,dk,dv] fp32 at slots[n] becomes the state after node last[n]
    (int32 CUDA tensor, within the tree; -1: it stays). With x [T,D] (the
    Conv1d's inputs) and win_pool [n_slots,4,D] fp32 the windows take the path's
    inputs likewise. Returns state_pool."""
    return _tree_commit("gla_tree_commit", k, v, log_lambda, False, cu_nodes, parents, last, state_pool, slots, x,
                        win_pool, stream)


def gla_tree_commit_gated(k, v, g, cu_nodes, parents, last, state_pool, slots=None, *, x=None, win_pool=None,
                          stream=None):
    """gla_tree_commit with a decay per node: g [T,H] fp32, as gla_tree_fwd_gated."""
    return _tree_commit("gla_tree_commit_gated", k, v, g, True, cu_nodes, parents, last, state_pool, slots, x, win_pool,
                        stream)


def gla_conv1d_tree(x, w, b, cu_nodes, parents, win_pool, slots=None, *, y=None, stream=None):
    """The causal Conv1d with SiLU along each path of the trees of gla_tree_fwd:
    x [T,D], w [D,4], b [D] or None; behind a tree's root the inputs of
    win_pool [n_slots,4,D] fp32 at slots[n], which stays as it is. Returns y [T,D]."""
    T, D = wide = _lead(x, 2, "x")
    c = _Quick(x, stream)
    index, dtype, i32, f32, cu = c.index, x.dtype, c.torch.int32, c.torch.float32, _offsets(cu_nodes)
    nseq, n_slots = cu[0] - 1, _lead(win_pool, 3, "win_pool")[0]
    args = (*_rows(x, dtype, wide, index, "x"), _at(w, f32, (D, 4), index, "w"), _at(b, f32, (D,), index, "b"),
            _at(cu_nodes, i32, cu, index, "cu_nodes"), _at(parents, i32, (T,), index, "parents"),
            _at(slots, i32, (nseq,), index, "slots"), _at(win_pool, f32, (n_slots, 4, D), index, "win_pool"), n_slots,
            nseq, T, D, _dtype_code(x))
    if y is None:
        y = c.empty(wide, dtype)
    c.run("gla_conv1d_tree", *args, _at(y, dtype, wide, index, "y"))
    return y


class _PagesCall(_Quick):
    """A call over pools of any element type, one or a sequence of [n_slots, ...] tensors."""

    __slots__ = ("pools",)

    def __init__(self, pools, stream):
        pools = [pools] if isinstance(pools, _torch().Tensor) else list(pools)
        if not pools:
            raise GlaError(GLA_ERR_INVALID_ARG, "argument", "no pools")
        super().__init__(pools[0], stream, element=False)
        index, n, k = self.index, (pools[0].shape or (0,))[0], len(pools)
        where, size = (_vp * k)(), (_ll * k)()
        for i, t in enumerate(pools):
            shape = t.shape
            if not shape or shape[0] != n or t.get_device() != index or not t.is_contiguous():
                raise GlaError(GLA_ERR_INVALID_ARG, "argument",
                               "pools must be contiguous, on one device and of as many pages each")
            where[i] = t.data_ptr()
            size[i] = t.nbytes // n if n else 4
        self.pools = (where, size, k, n)


def gla_pages_copy(pools, src, dst, *, stream=None):
    """Copies pages of the pools (a tensor [n_slots, ...] or several, of any
    type, as many pages each): page dst[i] becomes page src[i] (int32 CUDA
    tensors), in every pool. A source may have several targets (one prompt
    continued several times); targets are distinct and no other pair's source."""
    c = _PagesCall(pools, stream)
    n, i32 = _lead(src, 1, "src"), c.torch.int32
    c.run("gla_pages_copy", *c.pools, _at(src, i32, n, c.index, "src"), _at(dst, i32, n, c.index, "dst"), n[0])


def gla_pages_clear(pools, slots, *, stream=None):
    """Fills the pages `slots` (int32 CUDA tensor) of the pools with zeros, as a
    new sequence needs them; pools as gla_pages_copy."""
    c = _PagesCall(pools, stream)
    n = _lead(slots, 1, "slots")
    c.run("gla_pages_clear", *c.pools, _at(slots, c.torch.int32, n, c.index, "slots"), n[0])


def gla_pages_compact_workspace_size(n_slots) -> int:
    return int(lib().gla_pages_compact_workspace_size(n_slots))


def gla_pages_compact(pools, live, *, map=None, count=None, workspace=None, stream=None):
    """Moves the pages in use to the front of the pools (as gla_pages_copy):
    live [n_slots] bool or uint8 CUDA tensor. With L pages in use, those at L
    and above move into the free ones below, in ascending order. Returns (map
    [n_slots] int32: each page's new number, -1 where not in use; count [1]
    int32: L), on the device."""
    c = _PagesCall(pools, stream)
    n, index, i32, u8 = c.pools[3], c.index, c.torch.int32, c.torch.uint8
    kind = c.torch.bool if live.dtype == c.torch.bool else u8
    if map is None:
        map = c.empty((n,), i32)
    if count is None:
        count = c.empty((1,), i32)
    if workspace is None:
        need = gla_pages_compact_workspace_size(n)
        if need > 0:
            workspace = c.empty((need,), u8)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, "argument", "the workspace must be contiguous and on the call's device")
    scratch = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    c.run("gla_pages_compact", *c.pools, _at(live, kind, (n,), index, "live"), _at(map, i32, (n,), index, "map"),
          _at(count, i32, (1,), index, "count"), *scratch)
    return map, count


def gla_selftest_wait_timeout(limit_us=20000, *, stream=None):
    """Diagnostic: make the device-side bounded waits run out (no fault, no
    hang). Returns the int32 CUDA tensor [completed0, completed1, us_waited1];
    the next gla_check() raises GlaError(GLA_ERR_TIMEOUT)."""
    torch = _torch()
    result = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st = lib().gla_selftest_wait_timeout(int(limit_us), _ptr(result), _stream(stream))
    _raise_on(st, "gla_selftest_wait_timeout")
    return result[:3]


def gla_check(stream=None):
    """Synchronise the stream; raise GlaError on a CUDA error or a device-side timeout."""
    st = lib().gla_check(_stream(stream))
    _raise_on(st, "gla_check")
