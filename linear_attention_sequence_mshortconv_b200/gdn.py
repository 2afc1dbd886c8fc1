"""Thin Python binding of libkda's gated delta rule (see include/kda.h):

    S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   alpha_t = e^{g_t},
    o_t = S_t^T q_t,

with one gate per value head and Hv / Hk value heads to a query/key head.  ``forward`` and
``forward_varlen`` run whole sequences, ``backward`` and ``backward_varlen`` their gradients,
``step`` one token per request on a pool of states.

All tensors of a call are contiguous, on one CUDA device, and bf16 or fp32 alike (the states
are fp32).  A call runs on that device, on its current stream unless one is given, whichever
device is current.  There is no fallback: without ``libkda.so`` or a CUDA tensor it raises.
"""
from __future__ import annotations

import torch

from .kda import _check, _code, _cu_array, _dtype_code, load_library

# The current stream's handle without building a Stream object (some 3 us of a call whose
# kernel may take 5), and the current device; torch's public ways where a version lacks them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_Tensor = torch.Tensor


def check_tensors(first, named):
    """The tensors of a call, (name, tensor or None, shape, dtype), are contiguous CUDA tensors of the
    first one's device and of the shape and type given; None passes.  Returns the device's index."""
    if not isinstance(first, _Tensor) or not first.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    index = first.get_device()
    for name, t, shape, dtype in named:
        if t is None or (isinstance(t, _Tensor) and t.shape == shape and t.dtype is dtype
                         and t.get_device() == index and t.is_contiguous()):
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, q on {first.device}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must be contiguous")
    return index


def ptr(t):
    return None if t is None else t.data_ptr()


def empty(like, shape, dtype=torch.float32):
    """A contiguous tensor of another type on like's device (given its strides it takes the host half as long as
    from new_empty with a type)."""
    strides, step = [], 1
    for n in shape[::-1]:
        strides.append(step)
        step *= n or 1
    return torch.empty_strided(shape, strides[::-1], dtype=dtype, device=like.device)


def launch(index, stream, body):
    """body(stream handle) with the tensors' device and the launching stream current, so that what a
    call allocates belongs to the stream it runs on."""
    if stream is None:
        if _device() == index:
            return body(_raw_stream(index))
        with torch.cuda.device(index):
            return body(_raw_stream(index))
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def scratch(workspace, need, like):
    """(tensor, address, bytes): the caller's workspace, or one from torch's allocator."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != like.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need == 0:
        return None, None, 0
    t = empty(like, (need,), torch.uint8)
    return t, t.data_ptr(), need


def _sizes(q, v, tokens_dims):
    if not isinstance(q, _Tensor) or not isinstance(v, _Tensor) or q.ndim != tokens_dims + 2 or v.ndim != tokens_dims + 2:
        raise ValueError(f"q and v must have {tokens_dims + 2} dimensions")
    (*_, Hk, Dk), (*_, Hv, Dv) = q.shape, v.shape
    if Hk == 0 or Hv % Hk:
        raise ValueError(f"{Hv} value heads cannot share {Hk} query/key heads")
    return Hk, Hv, Dk, Dv


def _inputs(q, k, v, g, beta, lead, Hv):
    shape, gates, dtype = q.shape, (*lead, Hv), q.dtype
    return [("q", q, shape, dtype), ("k", k, shape, dtype), ("v", v, (*lead, *v.shape[-2:]), dtype),
            ("g", g, gates, dtype), ("beta", beta, gates, dtype)]


def _packed(cu_seqlens, T):
    arr, n = _cu_array(cu_seqlens)
    if n < 0 or int(arr[n]) > T:
        raise ValueError("cu_seqlens must end within the packed length")
    return arr, n


def workspace_size(B, T, Hk, Hv, Dk, Dv, dtype=torch.bfloat16) -> int:
    return int(load_library().gdn_forward_workspace_size(B, T, Hk, Hv, Dk, Dv, _code(dtype)))


def varlen_workspace_size(cu_seqlens, Hk, Hv, Dk, Dv, dtype=torch.bfloat16) -> int:
    arr, n = _cu_array(cu_seqlens)
    return int(load_library().gdn_forward_varlen_workspace_size(arr, n, Hk, Hv, Dk, Dv, _code(dtype)))


def backward_workspace_size(B, T, Hk, Hv, Dk, Dv, dtype=torch.bfloat16) -> int:
    return int(load_library().gdn_backward_workspace_size(B, T, Hk, Hv, Dk, Dv, _code(dtype)))


def backward_varlen_workspace_size(cu_seqlens, Hk, Hv, Dk, Dv, dtype=torch.bfloat16) -> int:
    arr, n = _cu_array(cu_seqlens)
    return int(load_library().gdn_backward_varlen_workspace_size(arr, n, Hk, Hv, Dk, Dv, _code(dtype)))


def _forward(q, k, v, g, beta, S0, lead, rows, seqs, need, o, S_T, want_state, workspace, stream, fn):
    Hk, Hv, Dk, Dv = _sizes(q, v, len(lead))
    dt = _dtype_code(q)
    state = (rows, Hv, Dk, Dv)
    index = check_tensors(q, _inputs(q, k, v, g, beta, lead, Hv) + [
        ("S0", S0, state, torch.float32), ("o", o, v.shape, q.dtype), ("S_T", S_T, state, torch.float32)])
    lib = load_library()

    def body(s):
        out = torch.empty_like(v) if o is None else o
        final = empty(q, state) if S_T is None and want_state else S_T
        keep, ws, ws_bytes = scratch(workspace, need(lib, Hk, Hv, Dk, Dv, dt), q)
        _check(fn, getattr(lib, fn)(ptr(q), ptr(k), ptr(v), ptr(g), ptr(beta), ptr(S0), ptr(out), ptr(final), *seqs,
                                    Hk, Hv, Dk, Dv, dt, ws, ws_bytes, s))
        return out, final

    return launch(index, stream, body)


def forward(q, k, v, g, beta, S0=None, *, o=None, S_T=None, want_state: bool = True, workspace=None, stream=None):
    """gdn_forward: q, k [B,T,Hk,Dk]; v [B,T,Hv,Dv]; g = ln(alpha), beta [B,T,Hv]; S0 [B,Hv,Dk,Dv]
    fp32 or None (zeros).  Returns (o [B,T,Hv,Dv], S_T [B,Hv,Dk,Dv] fp32 or None)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B,T,Hk,Dk]")
    B, T = q.shape[:2]
    return _forward(q, k, v, g, beta, S0, (B, T), B, (B, T),
                    lambda lib, Hk, Hv, Dk, Dv, dt: lib.gdn_forward_workspace_size(B, T, Hk, Hv, Dk, Dv, dt),
                    o, S_T, want_state, workspace, stream, "gdn_forward")


def forward_varlen(q, k, v, g, beta, cu_seqlens, S0=None, *, o=None, S_T=None, want_state: bool = True,
                   workspace=None, stream=None):
    """gdn_forward_varlen: packed samples on one token axis ([T_total, ...] tensors), the state
    restarting at every sample from its S0 [n,Hv,Dk,Dv] (None: zeros).  cu_seqlens: host sequence
    of n + 1 offsets; tokens behind the last offset are left as they are in a given o.  Returns
    (o [T_total,Hv,Dv], S_T [n,Hv,Dk,Dv] fp32 or None)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [T_total,Hk,Dk]")
    arr, n = _packed(cu_seqlens, q.shape[0])
    return _forward(q, k, v, g, beta, S0, (q.shape[0],), n, (arr, n),
                    lambda lib, Hk, Hv, Dk, Dv, dt: lib.gdn_forward_varlen_workspace_size(arr, n, Hk, Hv, Dk, Dv, dt),
                    o, S_T, want_state, workspace, stream, "gdn_forward_varlen")


def _backward(q, k, v, g, beta, do, S0, dS_T, lead, rows, seqs, need, want_dS0, workspace, stream, out, fn):
    Hk, Hv, Dk, Dv = _sizes(q, v, len(lead))
    dt = _dtype_code(q)
    state = (rows, Hv, Dk, Dv)
    grads = [("dq", q.shape), ("dk", q.shape), ("dv", v.shape), ("dg", (*lead, Hv)), ("dbeta", (*lead, Hv))]
    given = (None,) * 6 if out is None else tuple(out)
    index = check_tensors(q, _inputs(q, k, v, g, beta, lead, Hv) + [
        ("do", do, v.shape, q.dtype), ("S0", S0, state, torch.float32), ("dS_T", dS_T, state, torch.float32)] + [
        (name, t, shape, q.dtype) for (name, shape), t in zip(grads, given)] + [("dS0", given[5], state, torch.float32)])
    if out is not None and any(t is None for t in given[:5]):
        raise ValueError("out must hold dq, dk, dv, dg, dbeta and dS0 or None")
    lib = load_library()

    def body(s):
        d = given
        if out is None:
            d = (*(torch.empty_like(t) for t in (q, k, v, g, beta)),
                 empty(q, state) if want_dS0 else None)
        keep, ws, ws_bytes = scratch(workspace, need(lib, Hk, Hv, Dk, Dv, dt), q)
        _check(fn, getattr(lib, fn)(ptr(q), ptr(k), ptr(v), ptr(g), ptr(beta), ptr(S0), ptr(do), ptr(dS_T),
                                    *map(ptr, d), *seqs, Hk, Hv, Dk, Dv, dt, ws, ws_bytes, s))
        return d

    return launch(index, stream, body)


def backward(q, k, v, g, beta, do, S0=None, dS_T=None, *, want_dS0: bool = True, workspace=None, stream=None,
             out=None):
    """gdn_backward: (dq, dk, dv, dg, dbeta, dS0 or None) for dL/do = do and dL/dS_T = dS_T through
    forward(q, k, v, g, beta, S0); the gradients have the inputs' shapes and type, dS0 is fp32.
    `out` may hold preallocated tensors in that order."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B,T,Hk,Dk]")
    B, T = q.shape[:2]
    return _backward(q, k, v, g, beta, do, S0, dS_T, (B, T), B, (B, T),
                     lambda lib, Hk, Hv, Dk, Dv, dt: lib.gdn_backward_workspace_size(B, T, Hk, Hv, Dk, Dv, dt),
                     want_dS0, workspace, stream, out, "gdn_backward")


def backward_varlen(q, k, v, g, beta, do, cu_seqlens, S0=None, dS_T=None, *, want_dS0: bool = True, workspace=None,
                    stream=None, out=None):
    """gdn_backward_varlen: backward() over packed samples, as in forward_varlen()."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [T_total,Hk,Dk]")
    arr, n = _packed(cu_seqlens, q.shape[0])
    return _backward(q, k, v, g, beta, do, S0, dS_T, (q.shape[0],), n, (arr, n),
                     lambda lib, Hk, Hv, Dk, Dv, dt: lib.gdn_backward_varlen_workspace_size(arr, n, Hk, Hv, Dk, Dv, dt),
                     want_dS0, workspace, stream, out, "gdn_backward_varlen")


def step(q, k, v, g, beta, state, slots=None, *, o=None, stream=None):
    """gdn_step: one token of each of n requests.  q, k [n,Hk,Dk]; v [n,Hv,Dv]; g, beta [n,Hv];
    state [n_slots,Hv,Dk,Dv] fp32, updated in place; slots: int32 CUDA tensor [n] (None: request i
    uses state i), negative for a padding request.  Returns o [n,Hv,Dv] (zeros for padding).  A slot
    outside the pool, or named twice, is reported by the library's last device error."""
    Hk, Hv, Dk, Dv = _sizes(q, v, 1)
    dt = _dtype_code(q)
    n = q.shape[0]
    for name, t in (("k", k), ("g", g), ("beta", beta)):
        if t is None:
            raise TypeError(f"{name} must be a CUDA tensor")
    if not isinstance(state, _Tensor) or state.ndim != 4:
        raise ValueError("state must be [n_slots,Hv,Dk,Dv]")
    n_slots = state.shape[0]
    index = check_tensors(q, _inputs(q, k, v, g, beta, (n,), Hv) + [
        ("state", state, (n_slots, Hv, Dk, Dv), torch.float32), ("slots", slots, (n,), torch.int32),
        ("o", o, (n, Hv, Dv), q.dtype)])
    lib = load_library()

    def body(s):
        out = torch.empty_like(v) if o is None else o
        _check("gdn_step", lib.gdn_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                        state.data_ptr(), ptr(slots), out.data_ptr(), n, n_slots, Hk, Hv, Dk, Dv,
                                        dt, s))
        return out

    return launch(index, stream, body)
