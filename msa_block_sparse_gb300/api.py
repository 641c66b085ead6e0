"""Python binding of libmsa.so (ctypes, and csrc/binding.cpp for the calls of a
decode loop).  Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  Function names match the C ABI in include/msa.h; tensors
are torch CUDA tensors in the layouts that header states, outputs and workspaces are
allocated with torch when the caller does not pass them, and the work is enqueued
on the current stream.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmsa.so")

D = 128
TOPK = 16

_c_int, _c_float, _c_size, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
_c_double = ctypes.c_double

# name -> (restype, argtypes); mirrors include/msa.h
_SIGNATURES = {
    "msa_abi_version": (_c_int, []),
    "msa_last_error": (ctypes.c_char_p, []),
    "msa_check_status": (_c_int, [_vp]),
    "msa_selftest_wait": (_c_int, [_vp]),
    "msa_trace_begin": (_c_int, []),
    "msa_trace_end": (_c_int, [ctypes.c_char_p, _c_size]),
    "msa_qk_norm_rope": (_c_int, [_vp, _vp, _c_int, _c_int, _vp, _vp, _c_int, _c_int, _c_float,
                                  _c_float, _vp]),
    "msa_qk_norm_rope4": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _vp, _vp, _vp, _vp,
                                   _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                   _c_float, _c_float, _vp]),
    "msa_qk_norm_rope_bwd_workspace_size": (_c_size, [_c_int, _c_int]),
    "msa_qk_norm_rope_bwd": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _c_int,
                                      _c_int, _c_float, _c_float, _vp, _c_size, _vp]),
    "msa_decode_append": (_c_int, [_vp] * 14 + [_c_int] * 6 + [_c_float, _c_float, _vp, _vp, _vp]),
    "msa_index_select_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "msa_index_select": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp,
                                  _vp, _c_size, _vp]),
    "msa_index_select_ex": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                     _c_int, _vp, _vp, _c_size, _vp]),
    "msa_sparse_attn_fwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "msa_sparse_attn_fwd": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                     _c_int, _c_float, _vp, _vp, _vp, _c_size, _vp]),
    "msa_sparse_attn_fwd_train": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                           _c_int, _c_float, _vp, _vp, _vp, _c_size, _vp, _c_size,
                                           _vp]),
    "msa_sparse_attn_bwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "msa_sparse_attn_bwd": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int,
                                     _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp,
                                     _c_size, _vp]),
    "msa_sparse_attn_bwd_prepare": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_size,
                                             _vp]),
    "msa_sparse_attn_bwd_prepared": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int,
                                              _c_int, _c_int, _c_int, _c_int, _c_float, _vp, _vp,
                                              _vp, _vp, _c_size, _vp]),
    "msa_qsa_attn_fwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "msa_qsa_attn_fwd": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                  _c_int, _c_int, _c_float, _vp, _vp, _vp, _c_size, _vp]),
    "msa_qsa_attn_bwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "msa_qsa_attn_bwd": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int,
                                  _c_int, _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp,
                                  _c_size, _vp]),
    "msa_decode_step_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "msa_decode_step": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                 _c_int, _c_int, _c_float, _vp, _vp, _vp, _c_size, _vp]),
    "msa_decode_step_ex": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_float, _c_int, _vp, _vp, _vp, _c_size,
                                    _vp]),
    "msa_rope_init": (_c_int, [_vp, _c_int, _c_double, _c_int, _c_int] + [_c_double] * 5),
    "msa_qk_norm_rope_ex": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _c_int, _vp,
                                     _c_float, _vp]),
    "msa_qk_norm_rope_bwd_ex_workspace_size": (_c_size, [_c_int] * 3),
    "msa_qk_norm_rope_bwd_ex": (_c_int, [_vp] * 4 + [_c_int] * 3 + [_vp] * 3 + [_c_int, _vp,
                                                                             _c_float, _vp,
                                                                             _c_size, _vp]),
    "msa_cache4_store": (_c_int, [_vp] * 9 + [_c_int] * 5 + [_c_float] * 3 + [_vp]),
    "msa_cache4_load": (_c_int, [_vp] * 6 + [_c_int] * 5 + [_c_float] * 3 + [_vp] * 4),
    "msa_decode4_append": (_c_int, [_vp] * 14 + [_c_int] * 5 + [_vp] + [_c_float] * 4 + [_vp] * 3),
    "msa_decode4_step_workspace_size": (_c_size, [_c_int] * 4),
    "msa_decode4_step": (_c_int, [_vp] * 7 + [_c_int] * 5 + [_c_float] * 3 + [_c_int, _vp, _vp, _vp,
                                                                          _c_size, _vp]),
    "msa_pages_fork": (_c_int, [_vp] * 3 + [_c_int] + [_vp] * 3 + [_c_int] * 3 + [_vp, _vp]),
    "msa_pages_free": (_c_int, [_vp] * 2 + [_c_int] + [_vp] * 3 + [_c_int] * 3 + [_vp, _vp]),
    "msa_pages_extend_workspace_size": (_c_size, [_c_int] * 2),
    "msa_pages_extend": (_c_int, [_vp] * 4 + [_c_int] * 3 + [_vp, _vp, _c_int, _vp, _vp, _c_size,
                                                          _vp]),
    "msa_pages_compact_workspace_size": (_c_size, [_c_int]),
    "msa_pages_compact": (_c_int, [_vp] * 3 + [_c_int] * 3 + [_vp, _vp, _c_int, _vp, _vp, _vp,
                                                           _c_size, _vp]),
    "msa_pages_copy": (_c_int, [_vp, _vp, _c_int, _c_int, _vp, _vp, _c_int, _vp]),
    "msa_decode_step_static": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int,
                                        _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp]),
}

STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_CUDA",
          4: "MSA_ERR_TIMEOUT", 5: "MSA_ERR_BOUNDS"}

_lib = None


class MSAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _check(code: int):
    if code != 0:
        raise MSAError(code, lib().msa_last_error().decode())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _req(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _workspace(size: int, device, ws: Optional[torch.Tensor]):
    if ws is not None:
        if ws.numel() * ws.element_size() < size:
            raise ValueError(f"workspace needs {size} bytes")
        return ws
    return torch.empty(max(size, 256), dtype=torch.uint8, device=device)


def msa_check_status(device=None) -> None:
    """Synchronizes the current stream and raises if a kernel reported a timeout
    or an out-of-range index since the last check."""
    s = torch.cuda.current_stream(device).cuda_stream
    _check(lib().msa_check_status(ctypes.c_void_p(s)))


# ------------------------------------------------------------------ prologue

def msa_selftest_wait(device=None) -> None:
    """Launch the diagnostic kernel whose bounded wait runs out (~2 s); the next
    msa_check_status raises MSAError (timeout)."""
    s = torch.cuda.current_stream(device).cuda_stream
    _check(lib().msa_selftest_wait(ctypes.c_void_p(s)))


def msa_trace_begin() -> None:
    """Start recording CUDA-event timings around every library kernel launch."""
    _check(lib().msa_trace_begin())


def msa_trace_end() -> dict:
    """Stop recording; {kernel: {"launches": n, "ms": total}} since msa_trace_begin."""
    buf = ctypes.create_string_buffer(1 << 16)
    _check(lib().msa_trace_end(buf, len(buf)))
    import json
    return json.loads(buf.value.decode())


def msa_qk_norm_rope(x, w, cu_seqlens, out: Optional[torch.Tensor] = None, rope_dim: int = 64,
                     rope_base: float = 1.0e7, eps: float = 1.0e-6):
    """x bf16 [T, H, 128] -> out (default: a new tensor; pass out=x for in place):
    gemma RMSNorm with weight w (bf16 [128]) then partial RoPE at each token's
    position in its sequence."""
    T, H = x.shape[0], x.shape[1]
    _req(x, "x", torch.bfloat16, (T, H, D))
    _req(w, "w", torch.bfloat16, (D,))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    out = torch.empty_like(x) if out is None else out
    _req(out, "out", torch.bfloat16, (T, H, D))
    S = cu_seqlens.numel() - 1
    _check(lib().msa_qk_norm_rope(_ptr(x), _ptr(out), T, H, _ptr(w), _ptr(cu_seqlens), S,
                                  rope_dim, rope_base, eps, _stream(x)))
    return out


def msa_qk_norm_rope_bwd(x, dy, w, cu_seqlens, dx: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None, rope_dim: int = 64,
                         rope_base: float = 1.0e7, eps: float = 1.0e-6,
                         workspace: Optional[torch.Tensor] = None):
    """Gradients of msa_qk_norm_rope: (dx bf16 [T, H, 128], dw fp32 [128]) from
    the prologue input x and dy = dL/dy (pass dx=dy to overwrite dy)."""
    T, H = x.shape[0], x.shape[1]
    _req(x, "x", torch.bfloat16, (T, H, D))
    _req(dy, "dy", torch.bfloat16, (T, H, D))
    _req(w, "w", torch.bfloat16, (D,))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    dx = torch.empty_like(x) if dx is None else dx
    _req(dx, "dx", torch.bfloat16, (T, H, D))
    dw = torch.empty(D, dtype=torch.float32, device=x.device) if dw is None else dw
    _req(dw, "dw", torch.float32, (D,))
    S = cu_seqlens.numel() - 1
    size = lib().msa_qk_norm_rope_bwd_workspace_size(T, H)
    ws = _workspace(size, x.device, workspace)
    _check(lib().msa_qk_norm_rope_bwd(_ptr(x), _ptr(dy), _ptr(dx), _ptr(dw), T, H, _ptr(w),
                                      _ptr(cu_seqlens), S, rope_dim, rope_base, eps, _ptr(ws),
                                      ws.numel(), _stream(x)))
    return dx, dw


def msa_qk_norm_rope4(q, k, q_idx, k_idx, w_q, w_k, w_qi, w_ki, cu_seqlens, outs=None,
                      rope_dim: int = 64, rope_base: float = 1.0e7, eps: float = 1.0e-6):
    """The prologue of q, k, index-q and index-k in one launch.  `outs` is a
    4-tuple of output tensors (default: new tensors; pass the inputs for in place)."""
    T = q.shape[0]
    Hq, Hkv, Hi = q.shape[1], k.shape[1], q_idx.shape[1]
    _req(q, "q", torch.bfloat16, (T, Hq, D))
    _req(k, "k", torch.bfloat16, (T, Hkv, D))
    _req(q_idx, "q_idx", torch.bfloat16, (T, Hi, D))
    _req(k_idx, "k_idx", torch.bfloat16, (T, Hi, D))
    for n, w in (("w_q", w_q), ("w_k", w_k), ("w_qi", w_qi), ("w_ki", w_ki)):
        _req(w, n, torch.bfloat16, (D,))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    if outs is None:
        outs = tuple(torch.empty_like(t) for t in (q, k, q_idx, k_idx))
    for o_, t, n in zip(outs, (q, k, q_idx, k_idx), ("q_out", "k_out", "q_idx_out", "k_idx_out")):
        _req(o_, n, torch.bfloat16, tuple(t.shape))
    S = cu_seqlens.numel() - 1
    _check(lib().msa_qk_norm_rope4(_ptr(q), _ptr(outs[0]), Hq, _ptr(k), _ptr(outs[1]), Hkv,
                                   _ptr(q_idx), _ptr(outs[2]), _ptr(k_idx), _ptr(outs[3]), Hi,
                                   _ptr(w_q), _ptr(w_k), _ptr(w_qi), _ptr(w_ki),
                                   _ptr(cu_seqlens), S, T, rope_dim, rope_base, eps,
                                   _stream(q)))
    return tuple(outs)


# ------------------------------------------------------------------ index select

def msa_index_select(q_idx, k_idx, cu_seqlens, max_seqlen: int, topk: int = TOPK,
                     out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, n_init: int = 0) -> torch.Tensor:
    """Selected blocks int32 [T, Hi, 16] (ascending, -1 padded).  n_init > 0 applies
    the init rule (msa_index_select_ex: the first n_init blocks are always kept)."""
    T, Hi = q_idx.shape[0], q_idx.shape[1]
    _req(q_idx, "q_idx", torch.bfloat16, (T, Hi, D))
    _req(k_idx, "k_idx", torch.bfloat16, (T, Hi, D))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    S = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((T, Hi, topk), dtype=torch.int32, device=q_idx.device)
    _req(out, "out", torch.int32, (T, Hi, topk))
    size = lib().msa_index_select_workspace_size(T, S, Hi, max_seqlen)
    ws = _workspace(size, q_idx.device, workspace)
    if n_init:
        _check(lib().msa_index_select_ex(_ptr(q_idx), _ptr(k_idx), _ptr(cu_seqlens), S, T, Hi,
                                         max_seqlen, topk, n_init, _ptr(out), _ptr(ws),
                                         ws.numel(), _stream(q_idx)))
    else:
        _check(lib().msa_index_select(_ptr(q_idx), _ptr(k_idx), _ptr(cu_seqlens), S, T, Hi,
                                      max_seqlen, topk, _ptr(out), _ptr(ws), ws.numel(),
                                      _stream(q_idx)))
    return out


# ------------------------------------------------------------------ attention

def msa_sparse_attn_fwd(q, k, v, sel, cu_seqlens, max_seqlen: int, scale: Optional[float] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        bwd_workspace: Optional[torch.Tensor] = None):
    """Block-sparse attention forward: (o bf16 [T, Hq, 128], lse fp32 [T, Hq]).
    With bwd_workspace (msa_sparse_attn_fwd_train): that backward workspace's
    accumulators are zeroed while the forward runs, for a following
    msa_sparse_attn_bwd(..., workspace=bwd_workspace, prepared=True)."""
    T, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    _req(q, "q", torch.bfloat16, (T, Hq, D))
    _req(k, "k", torch.bfloat16, (T, Hkv, D))
    _req(v, "v", torch.bfloat16, (T, Hkv, D))
    _req(sel, "sel", torch.int32, (T, Hkv, TOPK))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    S = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _req(out, "out", torch.bfloat16, (T, Hq, D))
    _req(lse, "lse", torch.float32, (T, Hq))
    size = lib().msa_sparse_attn_fwd_workspace_size(T, S, Hq, Hkv, max_seqlen)
    ws = _workspace(size, q.device, workspace)
    if bwd_workspace is None:
        _check(lib().msa_sparse_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(sel), _ptr(cu_seqlens),
                                         S, T, Hq, Hkv, max_seqlen, scale, _ptr(out), _ptr(lse),
                                         _ptr(ws), ws.numel(), _stream(q)))
    else:
        bsize = lib().msa_sparse_attn_bwd_workspace_size(T, S, Hq, Hkv, max_seqlen)
        bws = _workspace(bsize, q.device, bwd_workspace)
        _check(lib().msa_sparse_attn_fwd_train(_ptr(q), _ptr(k), _ptr(v), _ptr(sel),
                                               _ptr(cu_seqlens), S, T, Hq, Hkv, max_seqlen, scale,
                                               _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                               _ptr(bws), bws.numel(), _stream(q)))
    return out, lse


def msa_sparse_attn_bwd_prepare(q, k, cu_seqlens, max_seqlen: int, workspace: torch.Tensor,
                                stream: Optional[torch.cuda.Stream] = None):
    """Clears the fp32 accumulators of `workspace` for one following
    msa_sparse_attn_bwd(..., prepared=True) of the same shapes (q [T, Hq, 128],
    k [T, Hkv, 128]), on `stream` (default: the current stream); the caller
    orders the two (an event when the streams differ)."""
    T, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    S = cu_seqlens.numel() - 1
    size = lib().msa_sparse_attn_bwd_workspace_size(T, S, Hq, Hkv, max_seqlen)
    ws = _workspace(size, q.device, workspace)
    st = ctypes.c_void_p((stream or torch.cuda.current_stream(q.device)).cuda_stream)
    _check(lib().msa_sparse_attn_bwd_prepare(T, S, Hq, Hkv, max_seqlen, _ptr(ws), ws.numel(), st))


def msa_sparse_attn_bwd(q, k, v, o, dout, lse, sel, cu_seqlens, max_seqlen: int,
                        scale: Optional[float] = None, dq=None, dk=None, dv=None,
                        workspace: Optional[torch.Tensor] = None, prepared: bool = False):
    """Block-sparse attention backward: (dq, dk, dv) in bf16.  prepared=True:
    `workspace` was cleared by msa_sparse_attn_bwd_prepare for this call."""
    T, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    _req(q, "q", torch.bfloat16, (T, Hq, D))
    _req(k, "k", torch.bfloat16, (T, Hkv, D))
    _req(v, "v", torch.bfloat16, (T, Hkv, D))
    _req(o, "o", torch.bfloat16, (T, Hq, D))
    _req(dout, "dout", torch.bfloat16, (T, Hq, D))
    _req(lse, "lse", torch.float32, (T, Hq))
    _req(sel, "sel", torch.int32, (T, Hkv, TOPK))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    S = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    size = lib().msa_sparse_attn_bwd_workspace_size(T, S, Hq, Hkv, max_seqlen)
    if prepared and workspace is None:
        raise ValueError("prepared=True needs the workspace that msa_sparse_attn_bwd_prepare cleared")
    ws = _workspace(size, q.device, workspace)
    call = lib().msa_sparse_attn_bwd_prepared if prepared else lib().msa_sparse_attn_bwd
    _check(call(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(sel),
                _ptr(cu_seqlens), S, T, Hq, Hkv, max_seqlen, scale, _ptr(dq), _ptr(dk), _ptr(dv),
                _ptr(ws), ws.numel(), _stream(q)))
    return dq, dk, dv


# ------------------------------------------------------------------ decode

def msa_decode_append(q, q_idx, k, v, k_idx, w_q, w_qi, w_k, w_ki, k_cache, v_cache,
                      kidx_cache, block_table, cache_lens, q_out=None, q_idx_out=None,
                      rope_dim: int = 64, rope_base: float = 1.0e7, eps: float = 1.0e-6):
    """Prologue of one new token per sequence (position cache_lens - 1), its k,
    index-k and v written into the paged caches in place; returns (q_out,
    q_idx_out) for msa_decode_step (pass q / q_idx to update them in place)."""
    B, Hq = q.shape[0], q.shape[1]
    P, Hkv = k_cache.shape[0], k_cache.shape[1]
    maxp = block_table.shape[1]
    _req(q, "q", torch.bfloat16, (B, Hq, D))
    for n, t in (("q_idx", q_idx), ("k", k), ("v", v), ("k_idx", k_idx)):
        _req(t, n, torch.bfloat16, (B, Hkv, D))
    for n, w in (("w_q", w_q), ("w_qi", w_qi), ("w_k", w_k), ("w_ki", w_ki)):
        _req(w, n, torch.bfloat16, (D,))
    for n, c in (("k_cache", k_cache), ("v_cache", v_cache), ("kidx_cache", kidx_cache)):
        _req(c, n, torch.bfloat16, (P, Hkv, 128, D))
    _req(block_table, "block_table", torch.int32, (B, maxp))
    _req(cache_lens, "cache_lens", torch.int32, (B,))
    q_out = torch.empty_like(q) if q_out is None else q_out
    q_idx_out = torch.empty_like(q_idx) if q_idx_out is None else q_idx_out
    _check(lib().msa_decode_append(_ptr(q), _ptr(q_idx), _ptr(k), _ptr(v), _ptr(k_idx),
                                   _ptr(w_q), _ptr(w_qi), _ptr(w_k), _ptr(w_ki), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(kidx_cache), _ptr(block_table),
                                   _ptr(cache_lens), B, Hq, Hkv, P, maxp, rope_dim, rope_base, eps,
                                   _ptr(q_out), _ptr(q_idx_out), _stream(q)))
    return q_out, q_idx_out


def msa_decode_step(q, q_idx, k_cache, v_cache, kidx_cache, block_table, cache_lens,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    sel_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, n_init: int = 0):
    """One decode step: (o bf16 [B, Hq, 128], sel int32 [B, Hkv, 16]).  n_init > 0
    applies the init rule (msa_decode_step_ex)."""
    B, Hq = q.shape[0], q.shape[1]
    P, Hkv = k_cache.shape[0], k_cache.shape[1]
    maxp = block_table.shape[1]
    _req(q, "q", torch.bfloat16, (B, Hq, D))
    _req(q_idx, "q_idx", torch.bfloat16, (B, Hkv, D))
    for n, c in (("k_cache", k_cache), ("v_cache", v_cache), ("kidx_cache", kidx_cache)):
        _req(c, n, torch.bfloat16, (P, Hkv, 128, D))
    _req(block_table, "block_table", torch.int32, (B, maxp))
    _req(cache_lens, "cache_lens", torch.int32, (B,))
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    if sel_out is None:
        sel_out = torch.empty((B, Hkv, TOPK), dtype=torch.int32, device=q.device)
    size = lib().msa_decode_step_workspace_size(B, Hq, Hkv, maxp)
    ws = _workspace(size, q.device, workspace)
    if n_init:
        _check(lib().msa_decode_step_ex(_ptr(q), _ptr(q_idx), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(kidx_cache), _ptr(block_table), _ptr(cache_lens), B,
                                        Hq, Hkv, P, maxp, scale, n_init, _ptr(out),
                                        _ptr(sel_out), _ptr(ws), ws.numel(), _stream(q)))
    else:
        _check(lib().msa_decode_step(_ptr(q), _ptr(q_idx), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(kidx_cache), _ptr(block_table), _ptr(cache_lens), B,
                                     Hq, Hkv, P, maxp, scale, _ptr(out), _ptr(sel_out),
                                     _ptr(ws), ws.numel(), _stream(q)))
    return out, sel_out


# ------------------------------------------------------------------ narrow blocks

QSA_D = 256


def msa_qsa_attn_fwd(q, k, v, sel, cu_seqlens, max_seqlen: int, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Narrow-block (4-token) sparse attention forward, head dim 256, Hq = 12 Hkv:
    (o bf16 [T, Hq, 256], lse fp32 [T, Hq]).  sel int32 [T, Hkv, topk]."""
    T, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    topk = sel.shape[-1]
    _req(q, "q", torch.bfloat16, (T, Hq, QSA_D))
    _req(k, "k", torch.bfloat16, (T, Hkv, QSA_D))
    _req(v, "v", torch.bfloat16, (T, Hkv, QSA_D))
    _req(sel, "sel", torch.int32, (T, Hkv, topk))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    S = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(QSA_D) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _req(out, "out", torch.bfloat16, (T, Hq, QSA_D))
    _req(lse, "lse", torch.float32, (T, Hq))
    size = lib().msa_qsa_attn_fwd_workspace_size(T, S, Hq, Hkv, max_seqlen)
    ws = _workspace(size, q.device, workspace)
    _check(lib().msa_qsa_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(sel), _ptr(cu_seqlens), S, T,
                                  Hq, Hkv, topk, max_seqlen, scale, _ptr(out), _ptr(lse),
                                  _ptr(ws), ws.numel(), _stream(q)))
    return out, lse


def msa_qsa_attn_bwd(q, k, v, o, dout, lse, sel, cu_seqlens, max_seqlen: int,
                     scale: Optional[float] = None, dq=None, dk=None, dv=None,
                     workspace: Optional[torch.Tensor] = None):
    """Narrow-block sparse attention backward: (dq, dk, dv) in bf16."""
    T, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    topk = sel.shape[-1]
    _req(q, "q", torch.bfloat16, (T, Hq, QSA_D))
    _req(k, "k", torch.bfloat16, (T, Hkv, QSA_D))
    _req(v, "v", torch.bfloat16, (T, Hkv, QSA_D))
    _req(o, "o", torch.bfloat16, (T, Hq, QSA_D))
    _req(dout, "dout", torch.bfloat16, (T, Hq, QSA_D))
    _req(lse, "lse", torch.float32, (T, Hq))
    _req(sel, "sel", torch.int32, (T, Hkv, topk))
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    S = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(QSA_D) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    size = lib().msa_qsa_attn_bwd_workspace_size(T, S, Hq, Hkv, max_seqlen)
    ws = _workspace(size, q.device, workspace)
    _check(lib().msa_qsa_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                  _ptr(sel), _ptr(cu_seqlens), S, T, Hq, Hkv, topk, max_seqlen,
                                  scale, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(),
                                  _stream(q)))
    return dq, dk, dv


# ------------------------------------------------------------------ prologue, any rotary layout

class Rope(ctypes.Structure):
    """A rotation (msa_rope_t): `dim` rotated channels, `layout` (0 half, 1
    interleaved), `gain` of the rotated channels and the angle per position of each
    pair.  Made by msa_rope; may be kept and used by any number of calls."""
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("gain", _c_float),
                ("reserved", _c_float), ("freqs", _c_double * 128)]


_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def msa_rope(dim: int = 64, base: float = 1.0e7, layout: str = "half", scaling: str = "none",
             factor: float = 1.0, orig_len: float = 32768.0, beta_fast: float = 32.0,
             beta_slow: float = 1.0, gain: Optional[float] = None) -> Rope:
    """The rotation of the first `dim` channels (msa_rope_init, host only): layout
    "half" or "interleaved", scaling "none", "linear", "ntk" or "yarn" by `factor` (yarn
    also takes the trained length and its two turn counts); gain None = the scaling's own."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    if gain is not None and not gain > 0:
        raise ValueError("gain must be > 0")
    r = Rope()
    _check(lib().msa_rope_init(ctypes.byref(r), dim, base, _LAYOUTS[layout], _SCALINGS[scaling],
                               factor, orig_len, beta_fast, beta_slow,
                               0.0 if gain is None else gain))
    return r


_binding = None


def _native():
    """The native part of the binding (csrc/binding.cpp): argument checks, outputs and
    the C call in one step.  Raises if it has not been built (there is no fallback)."""
    global _binding
    if _binding is None:
        lib()
        try:
            from . import _msa_torch
        except ImportError as e:
            raise RuntimeError("the native binding is missing or does not load: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        _binding = _msa_torch
    return _binding


def _rope_at(rope) -> int:
    if not isinstance(rope, Rope):
        raise ValueError("rope must come from msa_rope")
    return ctypes.addressof(rope)


def msa_qk_norm_rope_ex(x, w, rope: Rope, cu_seqlens: Optional[torch.Tensor] = None,
                        positions: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, eps: float = 1.0e-6):
    """x bf16 [T, H, D] (D 64, 128 or 256) -> out: gemma RMSNorm with weight w (bf16
    [D]; None: no norm), then the rotation `rope` at positions (int32 [T]) or at the
    tokens' places in cu_seqlens' sequences (tokens outside those are left alone).  Pass
    out=x for in place."""
    return _native().qk_norm_rope_ex(x, w, _rope_at(rope), cu_seqlens, positions, out, eps)


def msa_qk_norm_rope_bwd_ex(x, dy, w, rope: Rope, cu_seqlens: Optional[torch.Tensor] = None,
                            positions: Optional[torch.Tensor] = None,
                            dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                            eps: float = 1.0e-6, workspace: Optional[torch.Tensor] = None):
    """Gradients of msa_qk_norm_rope_ex: (dx bf16 [T, H, D], dw fp32 [D]) from its input
    x and dy (pass dx=dy to overwrite dy); with w None (dx, None), and x may be None."""
    return _native().qk_norm_rope_bwd_ex(x, dy, w, _rope_at(rope), cu_seqlens, positions, dx, dw, eps,
                                         workspace)


# ------------------------------------------------------------------ 4-bit paged cache

SLAB4 = 9216     # bytes of a page of one head: 128 x 64 of codes, 128 x 8 of scales
_SCALE = 1.0 / math.sqrt(D)


def _gains(gains):
    if len(gains) != 3:
        raise ValueError("gains must be those of k, v and k_idx")
    return gains


def msa_cache4_store(k, v, k_idx, k_cache, v_cache, kidx_cache, block_table, cu_seqlens,
                     start: Optional[torch.Tensor] = None, gains=(1.0, 1.0, 1.0)) -> None:
    """Writes a pack (k, v, k_idx bf16 [T, Hkv, 128], post-prologue) into 4-bit caches
    (uint8 [num_pages, Hkv, 9216]): token i of sequence s at position start[s] + i of
    row s of block_table.  k, v or k_idx may be None together with its cache.  gains:
    of k, v and k_idx, powers of two; the same ones have to be given when reading."""
    _native().cache4_store(k, v, k_idx, k_cache, v_cache, kidx_cache, block_table, cu_seqlens, start,
                           *_gains(gains))


def msa_cache4_load(k_cache, v_cache, kidx_cache, block_table, cu_seqlens, T: int,
                    start: Optional[torch.Tensor] = None, gains=(1.0, 1.0, 1.0), k=None, v=None,
                    k_idx=None):
    """The held values of a pack's positions, as bf16 [T, Hkv, 128] each: the inverse of
    msa_cache4_store.  A cache that is None is left out (its result is None)."""
    return _native().cache4_load(k_cache, v_cache, kidx_cache, block_table, cu_seqlens, T, start,
                                 *_gains(gains),
                                 k, v, k_idx)


def msa_decode4_append(q, q_idx, k, v, k_idx, w_q, w_qi, w_k, w_ki, k_cache, v_cache, kidx_cache,
                       block_table, cache_lens, rope: Rope, gains=(1.0, 1.0, 1.0), q_out=None,
                       q_idx_out=None, eps: float = 1.0e-6):
    """msa_decode_append into 4-bit caches: the prologue (norm, rotation `rope`) of one
    new token per sequence at position cache_lens - 1, its k, index-k and v held in 4
    bits; returns (q_out, q_idx_out).  Rows of length 0 are padding and left alone."""
    return _native().decode4_append(q, q_idx, k, v, k_idx, w_q, w_qi, w_k, w_ki, k_cache, v_cache,
                                    kidx_cache, block_table, cache_lens, _rope_at(rope), *_gains(gains),
                                    q_out, q_idx_out, eps)


def msa_decode4_step(q, q_idx, k_cache, v_cache, kidx_cache, block_table, cache_lens,
                     scale: Optional[float] = None, gains=(1.0, 1.0, 1.0),
                     out: Optional[torch.Tensor] = None, sel_out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, n_init: int = 0):
    """msa_decode_step over 4-bit caches: (o bf16 [B, Hq, 128], sel int32 [B, Hkv, 16]),
    Hq = 1 .. 16 heads per KV head.  Rows of length 0 get o = 0, sel = -1."""
    k_gain, v_gain, _ = _gains(gains)
    return _native().decode4_step(q, q_idx, k_cache, v_cache, kidx_cache, block_table, cache_lens,
                                  _SCALE if scale is None else scale, k_gain, v_gain, out, sel_out,
                                  workspace, n_init)


# ------------------------------------------------------------------ pages of a cache

def msa_pages_fork(src, dst, block_table, cache_lens, ref_count,
                   keep: Optional[torch.Tensor] = None, forked: Optional[torch.Tensor] = None):
    """Row dst[i] (empty) shares the pages of the first keep[i] tokens (None: all) of
    row src[i]; tables, lengths and reference counts change in place.  Returns forked
    int32 [n]: the length given, -1 where the pair was refused."""
    return _native().pages_fork(src, dst, block_table, cache_lens, ref_count, keep, forked)


def msa_pages_free(rows, block_table, cache_lens, ref_count, keep: Optional[torch.Tensor] = None,
                   dropped: Optional[torch.Tensor] = None):
    """Row rows[i] keeps its first keep[i] tokens (None: none); pages that no row
    holds any more are free.  Returns dropped int32 [n]: tokens dropped, -1 where refused."""
    return _native().pages_free(rows, block_table, cache_lens, ref_count, keep, dropped)


def msa_pages_extend(add, block_table, cache_lens, ref_count, caches,
                     done: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Row b grows by add[b] tokens: new pages from the free ones, and an own copy of a
    shared, partly filled last page in every tensor of `caches` (first dimension =
    pages, any format).  Returns done int32 [B]: 1 where the row has grown, 0 where the
    pool or the table is too small for it."""
    return _native().pages_extend(add, block_table, cache_lens, ref_count, caches, done, workspace)


def msa_pages_compact(block_table, cache_lens, ref_count, caches,
                      page_map: Optional[torch.Tensor] = None,
                      n_live: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None):
    """Moves the pages in use to the front of the pool, in every tensor of `caches`;
    tables and counts follow.  Returns (page_map int32 [num_pages], -1 for free pages,
    n_live int32 [1])."""
    return _native().pages_compact(block_table, cache_lens, ref_count, caches, page_map, n_live, workspace)


def msa_pages_copy(src, dst, caches) -> None:
    """Page src[i] -> page dst[i] in every tensor of `caches` (first dimension = pages)."""
    _native().pages_copy(src, dst, caches)


def workspace_bytes(call: str, *args) -> int:
    """Workspace size of `call` ('qk_norm_rope_bwd', 'index_select', 'sparse_attn_fwd',
    'sparse_attn_bwd', 'qsa_attn_fwd', 'qsa_attn_bwd', 'decode_step', 'qk_norm_rope_bwd_ex',
    'decode4_step', 'pages_extend', 'pages_compact') for the given sizes, as the C ABI
    reports it."""
    return int(getattr(lib(), f"msa_{call}_workspace_size")(*args))
