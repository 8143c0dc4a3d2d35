"""Binding of linear attention with a decay for each head (include/linear_attention.h).

Argument marshalling only, as in :mod:`.gated_delta`, whose conventions for devices, streams and
the memory of a call these functions share.

Shapes: q, k [B,T,Hk,K], v [B,T,Hv,V], one dtype (torch.bfloat16 or torch.float32); g float32 [Hv],
the log decay of each head; states float32 [B,Hv,V,K].  A packed batch of n sequences has B = 1 and
``cu_seqlens`` (int32 [n+1] on the device); its states are [n,Hv,V,K].  q, k and v may be slices of a
joint projection: dense in their last two dimensions, any stride from token to token that is a
multiple of 16 bytes.
"""
from __future__ import annotations

import ctypes

from . import wkv as _wkv
from .gated_delta import _check, _counts, _dense, _index, _On, _ptr, _token_stride
from .wkv import DT_BF16, DT_F32


class Problem(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("total", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
                ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong), ("slots_in", ctypes.c_void_p),
                ("slots_out", ctypes.c_void_p), ("pool", ctypes.c_int), ("scale", ctypes.c_float),
                ("dt", ctypes.c_int)]


_lib = None


def lib():
    """The built library with this module's functions declared (raises if it is not built)."""
    global _lib
    if _lib is None:
        L = _wkv.lib()
        vp, ci, sz, pp = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(Problem)
        for name, args, res in (
                ("linear_attention_forward", [pp] + [vp] * 8 + [sz, vp], ci),
                ("linear_attention_forward_workspace", [pp], sz),
                ("linear_attention_decode", [pp] + [vp] * 7, ci),
                ("linear_attention_backward", [pp] + [vp] * 13 + [sz, vp], ci),
                ("linear_attention_backward_workspace", [pp], sz)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def _problem(torch, q, k, v, g, cu_seqlens, slots_in, slots_out, pool, scale):
    """The C problem of checked inputs, and the shape of one sequence's states.  q [*lead, Hk, K] with
    lead (B, T), or (B,) for single tokens."""
    *lead, Hk, K = q.shape
    Hv, V = v.shape[-2:]
    dt, dev = q.dtype, q.device
    if dt == torch.bfloat16:
        code = DT_BF16
    elif dt == torch.float32:
        code = DT_F32
    else:
        raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")
    if dev.type != "cuda":
        raise ValueError("inputs must live on the GPU")
    if k.dtype != dt or v.dtype != dt:
        raise TypeError("q, k and v must share one dtype")
    if k.device != dev or v.device != dev:
        raise ValueError(f"all inputs must live on {dev}")
    _dense(g, "g", (Hv,), torch.float32, dev)
    n = lead[0]
    total = n * lead[1] if len(lead) == 2 else n
    cu = None
    if total >> 31:
        _counts(tokens=total)
    if cu_seqlens is not None:
        if n != 1:
            raise ValueError("a packed batch has B = 1")
        n = cu_seqlens.numel() - 1
        if n < 1:
            raise ValueError("cu_seqlens holds n + 1 offsets of n >= 1 sequences")
        _counts(sequences=n)
        cu = _index(torch, cu_seqlens, "cu_seqlens", n + 1, dev)
    into = _index(torch, slots_out, "slots", n, dev)
    start = into if slots_in is slots_out else _index(torch, slots_in, "slots_in", n, dev)
    p = Problem(n, total, cu, Hk, Hv, K, V, _token_stride(q, "q", lead, Hk, K),
                _token_stride(k, "k", lead, Hk, K), _token_stride(v, "v", lead, Hv, V), start, into,
                n if pool is None else pool, K ** -0.5 if scale is None else scale, code)
    return p, n, (Hv, V, K)


def _check_ranks(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k are [B,T,Hk,K], v is [B,T,Hv,V]")


def _query(name, tokens, Hk, Hv, K, V, sequences, packed, dtype):
    _counts(tokens=tokens, Hk=Hk, Hv=Hv, K=K, V=V, sequences=sequences)
    p = Problem(n_seq=sequences, total=tokens, Hk=Hk, Hv=Hv, K=K, V=V, pool=sequences,
                dt=_wkv._dtype_name_code(dtype))
    if packed:
        p.cu_seqlens = 16  # any address: sizes do not depend on the offsets
    return int(getattr(lib(), name)(ctypes.byref(p)))


def linear_attention_forward_workspace_bytes(tokens, Hk, Hv, K, V, *, sequences=1, packed=False,
                                             dtype="bf16") -> int:
    """Bytes of workspace of :func:`linear_attention_forward`."""
    return _query("linear_attention_forward_workspace", tokens, Hk, Hv, K, V, sequences, packed, dtype)


def linear_attention_backward_workspace_bytes(tokens, Hk, Hv, K, V, *, sequences=1, packed=False,
                                              dtype="bf16") -> int:
    """Bytes of workspace of :func:`linear_attention_backward`."""
    return _query("linear_attention_backward_workspace", tokens, Hk, Hv, K, V, sequences, packed, dtype)


def linear_attention_forward(q, k, v, g, s0=None, *, cu_seqlens=None, slots=None, slots_in=None,
                             scale=None, o=None, s_out=None, want_state=True, workspace=None,
                             stream=None):
    """linear_attention_forward: every token of every sequence.  Returns (o, s_out).

    Without ``slots``, s0 and s_out are [n,Hv,V,K] (s_out may be s0).  With ``slots`` (int32 [n] on
    the device) s0 and s_out are pools [slots,Hv,V,K], usually the same one: sequence i starts from
    state ``slots[i]`` of s0 (``slots_in[i]`` if that is given; -1: from zeros) and leaves its final
    state in ``slots[i]`` of s_out (-1: dropped), which then must be given.  ``scale`` is K^-0.5 by
    default.  Rows of a packed batch outside every sequence are not written (``o`` keeps what it held).
    It is a training step's forward too: :func:`linear_attention_backward` needs nothing but the inputs."""
    import torch

    pool = None
    if slots is not None or slots_in is not None:
        if slots is None:
            raise ValueError("slots_in comes with slots")
        if s_out is None and want_state:
            raise ValueError("with slots, the pool for the final states (s_out) must be given")
        ref = s0 if s0 is not None else s_out
        pool = 1 if ref is None else ref.shape[0]
        if slots_in is None:
            slots_in = slots
    _check_ranks(q, k, v)
    p, n, tail = _problem(torch, q, k, v, g, cu_seqlens, slots_in, slots, pool, scale)
    if slots is not None and s0 is None and s_out is None:
        p.slots_in = p.slots_out = None
        p.pool = n
    states = (p.pool, *tail)
    dev = q.device
    _dense(s0, "s0", states, torch.float32, dev)
    _dense(s_out, "s_out", states, torch.float32, dev)
    _dense(o, "o", v.shape, q.dtype, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, s0, o, s_out, cu_seqlens, slots, slots_in)
        if o is None:
            o = on.like(v)
        if s_out is None and want_state:
            s_out = on.empty(states, torch.float32) if s0 is None else on.like(s0)
        ref = ctypes.byref(p)
        workspace, size = on.workspace(lib().linear_attention_forward_workspace(ref), workspace)
        _check(lib().linear_attention_forward(
            ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s0), _ptr(o), _ptr(s_out), _ptr(workspace),
            size, on.handle), "linear_attention_forward")
    return o, s_out


def linear_attention_decode(q, k, v, g, state, *, slots=None, scale=None, o=None, stream=None):
    """linear_attention_decode: one token per sequence, q, k [B,Hk,K], v [B,Hv,V], g [Hv].  ``state``
    [B,Hv,V,K] float32, or a pool [slots,Hv,V,K] with ``slots`` (int32 [B] on the device; rows with a
    slot outside the pool are left as they are), is updated in place.  Returns o [B,Hv,V]."""
    import torch

    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k are [B,Hk,K], v is [B,Hv,V]")
    if state is None:
        raise ValueError("decode needs the state")
    pool = None if slots is None else state.shape[0]
    p, _, tail = _problem(torch, q, k, v, g, None, slots, slots, pool, scale)
    dev = q.device
    _dense(state, "state", (p.pool, *tail), torch.float32, dev)
    _dense(o, "o", v.shape, q.dtype, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, state, o, slots)
        if o is None:
            o = on.like(v)
        _check(lib().linear_attention_decode(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state), _ptr(o), on.handle),
            "linear_attention_decode")
    return o


def linear_attention_backward(q, k, v, g, d_o, s0=None, ds_T=None, *, cu_seqlens=None, scale=None,
                              grads=None, dg=None, want_dg=True, ds0=None, want_ds0=True,
                              workspace=None, stream=None):
    """linear_attention_backward.  Returns (dq, dk, dv, dg, ds0): the gradients of
    sum_t <o_t, d_o_t> + <S_T, ds_T> for the inputs of :func:`linear_attention_forward` (give the same
    s0, cu_seqlens and scale).  ``want_dg=False`` for decays that are not learned saves a fifth of
    a large call and returns None there; ``grads`` may pass the tensors for (dq, dk, dv); ``ds0`` may be
    ``ds_T`` (in place).  Rows of a packed batch outside every sequence are not written."""
    import torch

    _check_ranks(q, k, v)
    p, n, tail = _problem(torch, q, k, v, g, cu_seqlens, None, None, None, scale)
    dev, dt = q.device, q.dtype
    if d_o is None:
        raise ValueError("the backward needs d_o")
    _dense(d_o, "d_o", v.shape, dt, dev)
    for name, x in (("s0", s0), ("ds_T", ds_T), ("ds0", ds0)):
        _dense(x, name, (n, *tail), torch.float32, dev)
    _dense(dg, "dg", g.shape, torch.float32, dev)
    if grads is not None:
        if len(grads) != 3 or any(x is None for x in grads):
            raise ValueError("grads must hold the three gradient tensors (dq, dk, dv)")
        for name, x, like in zip(("dq", "dk", "dv"), grads, (q, k, v)):
            _dense(x, name, like.shape, dt, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, d_o, s0, ds_T, ds0, dg, cu_seqlens, *(grads or ()))
        if grads is None:
            grads = tuple(on.like(x) for x in (q, k, v))
        if dg is None and want_dg:
            dg = on.like(g)
        if ds0 is None and want_ds0:
            ds0 = on.empty((n, *tail), torch.float32)
        ref = ctypes.byref(p)
        workspace, size = on.workspace(lib().linear_attention_backward_workspace(ref), workspace)
        _check(lib().linear_attention_backward(
            ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(d_o), _ptr(s0), _ptr(ds_T),
            *(_ptr(x) for x in grads), _ptr(dg), _ptr(ds0), _ptr(workspace), size, on.handle),
            "linear_attention_backward")
    return (*grads, dg, ds0)
