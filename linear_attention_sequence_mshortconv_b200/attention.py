"""Thin Python binding of libkda's causal attention with grouped heads (see include/kda.h):

    o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j,   lse_i = ln sum_{j <= i} e^{scale q_i . k_j}

over rows or packed samples, H / Hkv query heads to a key/value head.  Tensors are contiguous, on
one CUDA device, and bf16 or fp32 alike (lse is fp32); a call runs on that device, on its current
stream unless one is given.  There is no fallback.
"""
from __future__ import annotations

import torch

from .gdn import _packed, check_tensors, empty, launch, ptr, scratch
from .kda import _check, _code, _dtype_code, load_library


def _sizes(q, k, dims):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.ndim != dims or k.ndim != dims:
        raise ValueError(f"q and k must have {dims} dimensions")
    (*_, H, D), Hkv = q.shape, k.shape[-2]
    if Hkv == 0 or H % Hkv:
        raise ValueError(f"{H} query heads cannot share {Hkv} key/value heads")
    return H, Hkv, D


def _forward(q, k, v, seqs, scale, o, lse, want_lse, stream, fn, dims):
    H, Hkv, D = _sizes(q, k, dims)
    dt = _dtype_code(q)
    shape, dtype = q.shape, q.dtype
    kv, rows = (*shape[:-2], Hkv, D), shape[:-1]
    index = check_tensors(q, [("q", q, shape, dtype), ("k", k, kv, dtype), ("v", v, kv, dtype), ("o", o, shape, dtype),
                              ("lse", lse, rows, torch.float32)])
    lib = load_library()

    def body(s):
        out = torch.empty_like(q) if o is None else o
        sums = empty(q, rows) if lse is None and want_lse else lse
        _check(fn, getattr(lib, fn)(ptr(q), ptr(k), ptr(v), ptr(out), ptr(sums), *seqs, H, Hkv, D,
                                    D ** -0.5 if scale is None else float(scale), dt, s))
        return out, sums

    return launch(index, stream, body)


def forward(q, k, v, *, scale=None, o=None, lse=None, want_lse: bool = True, stream=None):
    """attn_forward: q [B,T,H,D]; k, v [B,T,Hkv,D]; scale: 1/sqrt(D) unless given.  Returns
    (o [B,T,H,D], lse [B,T,H] fp32 or None)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B,T,H,D]")
    return _forward(q, k, v, tuple(q.shape[:2]), scale, o, lse, want_lse, stream, "attn_forward", 4)


def forward_varlen(q, k, v, cu_seqlens, *, scale=None, o=None, lse=None, want_lse: bool = True, stream=None):
    """attn_forward_varlen: packed samples on one token axis ([T_total, ...] tensors); cu_seqlens: host
    sequence of n + 1 offsets.  Tokens behind the last offset are left as they are in given outputs."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [T_total,H,D]")
    arr, n = _packed(cu_seqlens, q.shape[0])
    return _forward(q, k, v, (arr, n), scale, o, lse, want_lse, stream, "attn_forward_varlen", 3)


def backward_workspace_size(tokens, H, Hkv, D, dtype=torch.bfloat16) -> int:
    return int(load_library().attn_backward_workspace_size(tokens, H, Hkv, D, _code(dtype)))


def _backward(q, k, v, o, lse, do, seqs, tokens, scale, workspace, stream, out, fn, dims):
    H, Hkv, D = _sizes(q, k, dims)
    dt = _dtype_code(q)
    kv = (*q.shape[:-2], Hkv, D)
    given = (None,) * 3 if out is None else tuple(out)
    index = check_tensors(q, [("q", q, q.shape, q.dtype), ("k", k, kv, q.dtype), ("v", v, kv, q.dtype),
                              ("o", o, q.shape, q.dtype), ("lse", lse, q.shape[:-1], torch.float32), ("do", do, q.shape, q.dtype),
                              ("dq", given[0], q.shape, q.dtype), ("dk", given[1], kv, q.dtype), ("dv", given[2], kv, q.dtype)])
    if out is not None and any(t is None for t in given):
        raise ValueError("out must hold dq, dk and dv")
    if o is None or lse is None or do is None:
        raise ValueError("o, lse and do are needed")
    lib = load_library()

    def body(s):
        d = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)) if out is None else given
        keep, ws, ws_bytes = scratch(workspace, int(lib.attn_backward_workspace_size(tokens, H, Hkv, D, dt)), q)
        _check(fn, getattr(lib, fn)(ptr(q), ptr(k), ptr(v), ptr(o), ptr(lse), ptr(do), *map(ptr, d), *seqs, H, Hkv, D,
                                    D ** -0.5 if scale is None else float(scale), dt, ws, ws_bytes, s))
        return d

    return launch(index, stream, body)


def backward(q, k, v, o, lse, do, *, scale=None, workspace=None, stream=None, out=None):
    """attn_backward: (dq, dk, dv) for dL/do = do through forward(q, k, v), from the o and lse it
    returned; the gradients have the inputs' shapes and type.  `out` may hold preallocated tensors."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B,T,H,D]")
    return _backward(q, k, v, o, lse, do, tuple(q.shape[:2]), q.shape[0] * q.shape[1], scale, workspace, stream, out,
                     "attn_backward", 4)


def backward_varlen(q, k, v, o, lse, do, cu_seqlens, *, scale=None, workspace=None, stream=None, out=None):
    """attn_backward_varlen: backward() over packed samples, as in forward_varlen()."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [T_total,H,D]")
    arr, n = _packed(cu_seqlens, q.shape[0])
    return _backward(q, k, v, o, lse, do, (arr, n), int(arr[n]), scale, workspace, stream, out, "attn_backward_varlen", 3)
