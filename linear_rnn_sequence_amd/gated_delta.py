"""Binding of the gated delta rule and of the state moves (include/gated_delta.h).

Argument marshalling only, as in :mod:`.wkv`: the kernels of librwkv7_wkv.so do the work,
torch provides device memory and the stream.  Calls run on the tensors' device and, unless a
stream is given, on that device's current stream.  A given stream does not wait for the current
one, nor the other way round: the caller orders it behind what makes the inputs, and what reads
the results behind it.  The memory on both sides is safe to free at any time.

Shapes: q, k [B,T,Hk,K], v [B,T,Hv,V], g and beta [B,T,Hv] (g: log decay), one dtype
(torch.bfloat16 or torch.float32); states float32 [B,Hv,V,K].  A packed batch of n sequences has
B = 1 and ``cu_seqlens`` (int32 [n+1] on the device); its states are [n,Hv,V,K].  q, k and v may
be slices of a joint projection: dense in their last two dimensions, any stride from token to
token that is a multiple of 16 bytes.
"""
from __future__ import annotations

import ctypes

from . import wkv as _wkv
from .wkv import DT_BF16, DT_F32, Rwkv7Error

CHUNK = 64            # GATED_DELTA_CHUNK
STATE_MOVE_MAX = 1024


class Problem(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("total", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
                ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong), ("slots_in", ctypes.c_void_p),
                ("slots_out", ctypes.c_void_p), ("pool", ctypes.c_int), ("scale", ctypes.c_float),
                ("normalize", ctypes.c_int), ("dt", ctypes.c_int)]


_lib = None


def lib():
    """The built library with this module's functions declared (raises if it is not built)."""
    global _lib
    if _lib is None:
        L = _wkv.lib()
        vp, ci, sz, pp = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(Problem)
        for name, args, res in (
                ("gated_delta_forward", [pp] + [vp] * 9 + [sz, vp], ci),
                ("gated_delta_forward_workspace", [pp], sz),
                ("gated_delta_decode", [pp] + [vp] * 8, ci),
                ("gated_delta_forward_train", [pp] + [vp] * 11 + [sz, vp], ci),
                ("gated_delta_chunks", [pp], ci),
                ("gated_delta_backward", [pp] + [vp] * 16 + [sz, vp], ci),
                ("gated_delta_backward_workspace", [pp], sz),
                ("state_move", [vp, ci, sz, ci, sz, vp, vp, ci, vp], ci)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def _check(code, where):
    if code != 0:
        raise Rwkv7Error(code, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _counts(**counts):
    """Refuses numbers that the C interface's ints do not hold (ctypes would cut them off)."""
    for name, n in counts.items():
        if n >= 1 << 31:
            raise ValueError(f"{name}: {n} is not below 2^31")


def _token_stride(x, name, lead, H, C):
    """Elements from one token's channels to the next's (0: dense) of x [*lead, H, C]."""
    shape = (*lead, H, C)
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {shape}")
    if x.is_contiguous():
        return 0
    s = x.stride()
    B, T = lead if len(lead) == 2 else (1, *lead)
    step = s[-3] if T > 1 else s[0]
    if B * T <= 1:
        step = H * C
    if s[-1] != 1 or (H > 1 and s[-2] != C) or (B > 1 and s[0] != T * step) or step < H * C:
        raise ValueError(f"{name}: the channels of a token must be dense and tokens equally spaced, "
                         f"none in another's place (strides {s})")
    return step


def _dense(t, name, shape, dtype, device):
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, not {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ckpt_size(torch, V, K, dtype):
    """Elements from state to state of the stored ones (GATED_DELTA_CKPT_SIZE)."""
    return V * K + V * K // 4 if dtype == torch.bfloat16 else V * K


def _check_ckpt(torch, t, chunks, tail, dtype, device):
    """The states that the training forward stores: [chunks,Hv,V,K], GATED_DELTA_CKPT_SIZE apart with the
    further bits behind each, the last one as well; or all of it as [chunks,Hv,GATED_DELTA_CKPT_SIZE]."""
    Hv, V, K = tail
    size = _ckpt_size(torch, V, K, dtype)
    if t.dim() == 3:
        return _dense(t, "s_ckpt", (chunks, Hv, size), dtype, device)
    if t.shape != (chunks, *tail) or t.dtype != dtype or t.device != device:
        raise ValueError(f"s_ckpt: {tuple(t.shape)} {t.dtype} on {t.device}, expected {(chunks, *tail)} {dtype} "
                         f"on {device}")
    if chunks and (t.stride() != (Hv * size, size, K, 1) or t.untyped_storage().nbytes() <
                   (t.storage_offset() + chunks * Hv * size) * t.element_size()):
        raise ValueError("s_ckpt must be the tensor that gated_delta_forward_train returned")


def _index(torch, t, name, n, device):
    if t is None:
        return None
    _dense(t, name, (n,), torch.int32, device)
    return t.data_ptr()


def _problem(torch, q, k, v, g, beta, cu_seqlens, slots_in, slots_out, pool, scale, normalize):
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
        raise TypeError("all per-token inputs must share one dtype")
    if k.device != dev or v.device != dev:
        raise ValueError(f"all inputs must live on {dev}")
    gates = (*lead, Hv)
    _dense(g, "g", gates, dt, dev)
    _dense(beta, "beta", gates, dt, dev)
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
                n if pool is None else pool, K ** -0.5 if scale is None else scale,
                1 if normalize else 0, code)
    return p, n, (Hv, V, K)


def _check_ranks(q, k, v, g, beta):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or g.dim() != 3 or beta.dim() != 3:
        raise ValueError("q and k are [B,T,Hk,K], v is [B,T,Hv,V], g and beta are [B,T,Hv]")


class _On:
    """The tensors' device as the current one, and the stream a call goes to.  With a given stream, the
    call's memory belongs to it too: memory of the current stream may still be in use by what that
    stream has queued (its last owner was freed on the host), which the given one does not wait for."""

    __slots__ = ("torch", "device", "guard", "given", "caller", "handle")

    def __init__(self, torch, device, stream):
        index = device.index
        self.torch, self.device, self.given = torch, device, stream
        if stream is None:
            # the handle of torch.cuda.current_stream(device), without the object around it: 1.8 us of a
            # single token's 14
            self.handle = torch._C._cuda_getCurrentRawStream(index)
            self.guard = None if torch.cuda.current_device() == index else torch.cuda.device(device)
        elif stream.device == device:
            self.handle = stream.cuda_stream
            self.caller = torch.cuda.current_stream(device)
            self.guard = torch.cuda.stream(stream)  # its device too
        else:
            raise ValueError(f"the stream must be one of {device}, not {stream.device}")

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False

    def uses(self, *tensors):
        """The caller's tensors: freed after the call, their memory is not handed out again before a given
        stream's work is done."""
        if self.given is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.given)

    def empty(self, shape, dtype):
        """Memory for the caller: freed, it is not handed out again before the work that the caller's
        stream has queued by then is done either."""
        t = self.torch.empty(shape, dtype=dtype, device=self.device)
        if self.given is not None:
            t.record_stream(self.caller)
        return t

    def like(self, x):
        """Dense memory of x's shape and type."""
        if self.given is not None or not x.is_contiguous():
            return self.empty(x.shape, x.dtype)
        return self.torch.empty_like(x)

    def workspace(self, need, given):
        if given is None:  # the call's alone
            return self.torch.empty((need,), dtype=self.torch.uint8, device=self.device) if need else None, need
        if not given.is_contiguous() or given.device != self.device:
            raise ValueError(f"the workspace must be a contiguous tensor on {self.device}")
        self.uses(given)
        return given, given.numel() * given.element_size()


def _query(name, tokens, Hk, Hv, K, V, sequences, packed, dtype):
    _counts(tokens=tokens, Hk=Hk, Hv=Hv, K=K, V=V, sequences=sequences)
    p = Problem(n_seq=sequences, total=tokens, Hk=Hk, Hv=Hv, K=K, V=V, pool=sequences,
                dt=_wkv._dtype_name_code(dtype))
    if packed:
        p.cu_seqlens = 16  # any address: sizes do not depend on the offsets
    return int(getattr(lib(), name)(ctypes.byref(p)))


def gated_delta_forward_workspace_bytes(tokens, Hk, Hv, K, V, *, sequences=1, packed=False,
                                        dtype="bf16") -> int:
    """Bytes of workspace of :func:`gated_delta_forward` and of the training forward."""
    return _query("gated_delta_forward_workspace", tokens, Hk, Hv, K, V, sequences, packed, dtype)


def gated_delta_backward_workspace_bytes(tokens, Hk, Hv, K, V, *, sequences=1, packed=False,
                                         dtype="bf16") -> int:
    """Bytes of workspace of :func:`gated_delta_backward`."""
    return _query("gated_delta_backward_workspace", tokens, Hk, Hv, K, V, sequences, packed, dtype)


def gated_delta_chunks(tokens, *, sequences=1, packed=False) -> int:
    """Number of chunk states that the training forward stores."""
    return _query("gated_delta_chunks", tokens, 1, 1, 64, 64, sequences, packed, "bf16")


def gated_delta_ckpt_size(V, K, *, dtype="bf16") -> int:
    """Elements of one stored state (GATED_DELTA_CKPT_SIZE): V K, and in bf16 V K / 4 for its further bits."""
    return V * K + (V * K // 4 if _wkv._dtype_name_code(dtype) == DT_BF16 else 0)


def gated_delta_forward(q, k, v, g, beta, s0=None, *, cu_seqlens=None, slots=None, slots_in=None,
                        scale=None, normalize=False, o=None, s_out=None, want_state=True,
                        workspace=None, stream=None):
    """gated_delta_forward: every token of every sequence.  Returns (o, s_out).

    Without ``slots``, s0 and s_out are [n,Hv,V,K] (s_out may be s0).  With ``slots`` (int32 [n] on
    the device) s0 and s_out are pools [slots,Hv,V,K], usually the same one: sequence i starts from
    state ``slots[i]`` of s0 (``slots_in[i]`` if that is given; -1: from zeros) and leaves its final
    state in ``slots[i]`` of s_out (-1: dropped), which then must be given.  ``scale`` is K^-0.5 by
    default; ``normalize`` divides q and k by their norms.  Rows of a packed batch outside every
    sequence are not written (``o`` keeps what it held)."""
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
    _check_ranks(q, k, v, g, beta)
    p, n, tail = _problem(torch, q, k, v, g, beta, cu_seqlens, slots_in, slots, pool, scale, normalize)
    if slots is not None and s0 is None and s_out is None:
        p.slots_in = p.slots_out = None
        p.pool = n
    states = (p.pool, *tail)
    dev = q.device
    _dense(s0, "s0", states, torch.float32, dev)
    _dense(s_out, "s_out", states, torch.float32, dev)
    _dense(o, "o", v.shape, q.dtype, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, beta, s0, o, s_out, cu_seqlens, slots, slots_in)
        if o is None:
            o = on.like(v)
        if s_out is None and want_state:
            s_out = on.empty(states, torch.float32) if s0 is None else on.like(s0)
        ref = ctypes.byref(p)
        workspace, size = on.workspace(lib().gated_delta_forward_workspace(ref), workspace)
        _check(lib().gated_delta_forward(
            ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(s0), _ptr(o), _ptr(s_out),
            _ptr(workspace), size, on.handle), "gated_delta_forward")
    return o, s_out


def gated_delta_decode(q, k, v, g, beta, state, *, slots=None, scale=None, normalize=False, o=None,
                       stream=None):
    """gated_delta_decode: one token per sequence, q, k [B,Hk,K], v [B,Hv,V], g, beta [B,Hv].
    ``state`` [B,Hv,V,K] float32, or a pool [slots,Hv,V,K] with ``slots`` (int32 [B] on the device;
    rows with a slot outside the pool are left as they are), is updated in place.  Returns o [B,Hv,V]."""
    import torch

    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or g.dim() != 2 or beta.dim() != 2:
        raise ValueError("q and k are [B,Hk,K], v is [B,Hv,V], g and beta are [B,Hv]")
    if state is None:
        raise ValueError("decode needs the state")
    pool = None if slots is None else state.shape[0]
    p, _, tail = _problem(torch, q, k, v, g, beta, None, slots, slots, pool, scale, normalize)
    dev = q.device
    _dense(state, "state", (p.pool, *tail), torch.float32, dev)
    _dense(o, "o", v.shape, q.dtype, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, beta, state, o, slots)
        if o is None:
            o = on.like(v)
        _check(lib().gated_delta_decode(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(o),
            on.handle), "gated_delta_decode")
    return o


def gated_delta_forward_train(q, k, v, g, beta, s0=None, *, cu_seqlens=None, scale=None,
                              normalize=False, o=None, s_out=None, want_state=True, s_ckpt=None,
                              u=None, workspace=None, stream=None):
    """gated_delta_forward_train.  Returns (o, s_out, s_ckpt, u); s_ckpt [chunks,Hv,V,K] and u (like
    v), in the inputs' dtype, are what :func:`gated_delta_backward` needs besides the inputs.  bf16
    states have further bits behind each, which a copy of that view would lose (it is refused).  To
    move or copy them meanwhile (activation offload, hooks on saved tensors), give ``s_ckpt`` as a tensor
    [chunks,Hv,:func:`gated_delta_ckpt_size`], which holds them too and which the backward takes as well."""
    import torch

    _check_ranks(q, k, v, g, beta)
    p, n, tail = _problem(torch, q, k, v, g, beta, cu_seqlens, None, None, None, scale, normalize)
    dev = q.device
    ref = ctypes.byref(p)
    chunks = lib().gated_delta_chunks(ref)
    _dense(s0, "s0", (n, *tail), torch.float32, dev)
    _dense(s_out, "s_out", (n, *tail), torch.float32, dev)
    _dense(o, "o", v.shape, q.dtype, dev)
    if s_ckpt is not None:
        _check_ckpt(torch, s_ckpt, chunks, tail, q.dtype, dev)
    _dense(u, "u", v.shape, q.dtype, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, beta, s0, o, s_out, s_ckpt, u, cu_seqlens)
        o = on.like(v) if o is None else o
        u = on.like(v) if u is None else u
        if s_ckpt is None:
            Hv, V, K = tail
            size = _ckpt_size(torch, V, K, q.dtype)
            s_ckpt = on.empty((chunks * Hv * size,), q.dtype).as_strided((chunks, *tail), (Hv * size, size, K, 1))
        if s_out is None and want_state:
            s_out = on.empty((n, *tail), torch.float32) if s0 is None else on.like(s0)
        workspace, size = on.workspace(lib().gated_delta_forward_workspace(ref), workspace)
        _check(lib().gated_delta_forward_train(
            ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(s0), _ptr(o), _ptr(s_out),
            _ptr(s_ckpt), _ptr(u), _ptr(workspace), size, on.handle), "gated_delta_forward_train")
    return o, s_out, s_ckpt, u


def gated_delta_backward(q, k, v, g, beta, d_o, s_ckpt, u, ds_T=None, *, cu_seqlens=None, scale=None,
                         normalize=False, grads=None, ds0=None, want_ds0=True, workspace=None,
                         stream=None):
    """gated_delta_backward.  Returns (dq, dk, dv, dg, dbeta, ds0): the gradients of
    sum_t <o_t, d_o_t> + <S_T, ds_T> for the inputs of :func:`gated_delta_forward_train` (give the
    same scale and normalize).  ``grads`` may pass the five output tensors; ``ds0`` may be ``ds_T``
    (in place).  Rows of a packed batch outside every sequence are not written."""
    import torch

    _check_ranks(q, k, v, g, beta)
    p, n, tail = _problem(torch, q, k, v, g, beta, cu_seqlens, None, None, None, scale, normalize)
    dev, dt = q.device, q.dtype
    ref = ctypes.byref(p)
    _dense(d_o, "d_o", v.shape, dt, dev)
    if s_ckpt is not None:
        _check_ckpt(torch, s_ckpt, lib().gated_delta_chunks(ref), tail, dt, dev)
    _dense(u, "u", v.shape, dt, dev)
    _dense(ds_T, "ds_T", (n, *tail), torch.float32, dev)
    _dense(ds0, "ds0", (n, *tail), torch.float32, dev)
    if d_o is None or s_ckpt is None or u is None:
        raise ValueError("the backward needs d_o, s_ckpt and u")
    if grads is not None:
        if len(grads) != 5 or any(x is None for x in grads):
            raise ValueError("grads must hold the five gradient tensors (dq, dk, dv, dg, dbeta)")
        for name, x, like in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, (q, k, v, g, beta)):
            _dense(x, name, like.shape, dt, dev)
    with _On(torch, dev, stream) as on:
        on.uses(q, k, v, g, beta, d_o, s_ckpt, u, ds_T, ds0, cu_seqlens, *(grads or ()))
        if grads is None:
            grads = tuple(on.like(x) for x in (q, k, v, g, beta))
        if ds0 is None and want_ds0:
            ds0 = on.empty((n, *tail), torch.float32) if ds_T is None else on.like(ds_T)
        workspace, size = on.workspace(lib().gated_delta_backward_workspace(ref), workspace)
        _check(lib().gated_delta_backward(
            ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(d_o), _ptr(s_ckpt), _ptr(u),
            _ptr(ds_T), *(_ptr(x) for x in grads), _ptr(ds0), _ptr(workspace), size, on.handle),
            "gated_delta_backward")
    return (*grads, ds0)


def state_move(pool, src, dst, *, slot_dim=0, stream=None):
    """state_move: ``pool[dst[i]] = old pool[src[i]]`` for all i at once, zeros where src[i] is -1
    (copies, forks, reorders, compacts and frees states).  ``pool``: a tensor of any dtype with the
    slots along dimension ``slot_dim`` 0, or 1 for a pool [layers, slots, ...] whose layers all move;
    each layer is contiguous.  src, dst: int32 [n] on the pool's device, n <= 1024.  Pairs out of range
    are left out; of pairs with the same target the last counts.  Returns ``pool``."""
    import torch

    if slot_dim not in (0, 1) or pool.dim() <= slot_dim:
        raise ValueError("slot_dim is 0 or 1, a dimension of the pool")
    dev = pool.device
    if dev.type != "cuda":
        raise ValueError("the pool must live on the GPU")
    layers = pool.shape[0] if slot_dim else 1
    if layers < 1 or not (pool.is_contiguous() or (slot_dim and pool[0].is_contiguous())):
        raise ValueError("each layer's slots must be contiguous")
    slots = pool.shape[slot_dim]
    size = pool.element_size()
    for d in pool.shape[slot_dim + 1:]:
        size *= d
    n = src.numel()
    _counts(layers=layers, slots=slots, pairs=n)
    _index(torch, src, "src", n, dev)
    _index(torch, dst, "dst", n, dev)
    step = pool.stride(0) * pool.element_size() if slot_dim and layers > 1 else 0
    with _On(torch, dev, stream) as on:
        on.uses(pool, src, dst)
        _check(lib().state_move(_ptr(pool), layers, step, slots, size, _ptr(src), _ptr(dst), n, on.handle),
               "state_move")
    return pool
