"""Binding of the group norm with an activation or gate (include/group_norm.h).

Argument marshalling only, as in :mod:`.gated_delta`, whose conventions for devices, streams and
the memory of a call these functions share.

Shapes: x and gate [..., C] in one dtype (torch.bfloat16 or torch.float32), channels last, each row
(token) normalised by itself in ``groups`` groups of C / groups neighbouring channels; weight and
bias float32 [C].  x and gate may be slices of a joint projection: dense channels, rows equally
spaced, at most 2^23 elements from one to the next.  The readouts [B,T,Hv,V] of a recurrence are
``o.flatten(-2)`` with ``groups=Hv``.
"""
from __future__ import annotations

import ctypes

from . import wkv as _wkv
from .gated_delta import _check, _dense, _On, _ptr
from .wkv import DT_BF16, DT_F32

ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}
MAX_SIZE = 1024  # channels of a group


class Problem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("groups", ctypes.c_int), ("size", ctypes.c_int),
                ("x_stride", ctypes.c_longlong), ("gate_stride", ctypes.c_longlong), ("eps", ctypes.c_float),
                ("activation", ctypes.c_int), ("rms", ctypes.c_int), ("dt", ctypes.c_int)]


_lib = None


def lib():
    """The built library with this module's functions declared (raises if it is not built)."""
    global _lib
    if _lib is None:
        L = _wkv.lib()
        vp, ci, sz, pp = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(Problem)
        for name, args, res in (
                ("group_norm_forward", [pp] + [vp] * 6, ci),
                ("group_norm_backward", [pp] + [vp] * 10 + [sz, vp], ci),
                ("group_norm_backward_workspace", [pp], sz)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def _row_stride(x, name, shape):
    """Elements from one row's channels to the next's (0: dense) of x [..., C]."""
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.is_contiguous():
        return 0
    C = shape[-1]
    step, rows = 0, 1  # from row to row, and the rows that lie so
    for n, s in zip(reversed(shape[:-1]), reversed(x.stride()[:-1])):
        if n == 1:
            continue
        if rows > 1 and s != step * rows:
            raise ValueError(f"{name}: rows must be equally spaced (strides {x.stride()})")
        if rows == 1:
            step = s
        rows *= n
    if (C > 1 and x.stride(-1) != 1) or (rows > 1 and step < C):
        raise ValueError(f"{name}: the channels of a row must be dense and no row in another's place "
                         f"(strides {x.stride()})")
    return step if rows > 1 else C


def _problem(torch, x, groups, weight, bias, gate, activation, eps, rms):
    if x.dim() < 1:
        raise ValueError("x is [..., C]")
    dt, dev = x.dtype, x.device
    if dt == torch.bfloat16:
        code = DT_BF16
    elif dt == torch.float32:
        code = DT_F32
    else:
        raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")
    if dev.type != "cuda":
        raise ValueError("inputs must live on the GPU")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r}, expected one of {', '.join(ACTIVATIONS)}")
    C = x.shape[-1]
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"{C} channels are not {groups} equal groups")
    if C // groups > MAX_SIZE:
        raise ValueError(f"groups of {C // groups} channels, at most {MAX_SIZE}")
    _dense(weight, "weight", (C,), torch.float32, dev)
    _dense(bias, "bias", (C,), torch.float32, dev)
    gate_stride = 0
    if gate is not None:
        if gate.dtype != dt:
            raise TypeError(f"gate: dtype {gate.dtype}, expected {dt}")
        if gate.device != dev:
            raise ValueError(f"gate must live on {dev}, not {gate.device}")
        gate_stride = _row_stride(gate, "gate", x.shape)
    return Problem(x.numel() // C, groups, C // groups, _row_stride(x, "x", x.shape), gate_stride, eps,
                   ACTIVATIONS[activation], 1 if rms else 0, code)


def group_norm_backward_workspace_bytes(rows, groups, size, *, dtype="bf16") -> int:
    """Bytes of workspace of :func:`group_norm_backward` where weight's or bias' gradient is wanted."""
    if groups >= 1 << 31 or size >= 1 << 31:
        raise ValueError("groups and size are below 2^31")
    p = Problem(rows=rows, groups=groups, size=size, dt=_wkv._dtype_name_code(dtype))
    return int(lib().group_norm_backward_workspace(ctypes.byref(p)))


def group_norm_forward(x, groups, *, weight=None, bias=None, gate=None, activation="silu", eps=1e-5,
                       rms=False, y=None, stream=None):
    """group_norm_forward: n = (x - mean) / sqrt(var + eps) weight + bias per row and group (``rms``:
    x / sqrt(mean(x^2) + eps)), and y = n act(gate) with a gate, act(n) without one.  ``activation``
    is "none", "silu" or "sigmoid".  ``y`` may be a dense ``x`` (in place).  Returns y, dense, like x."""
    import torch

    p = _problem(torch, x, groups, weight, bias, gate, activation, eps, rms)
    _dense(y, "y", x.shape, x.dtype, x.device)
    with _On(torch, x.device, stream) as on:
        on.uses(x, weight, bias, gate, y)
        if y is None:
            y = on.like(x)
        _check(lib().group_norm_forward(ctypes.byref(p), _ptr(x), _ptr(gate), _ptr(weight), _ptr(bias), _ptr(y),
                                        on.handle), "group_norm_forward")
    return y


def group_norm_backward(x, groups, dy, *, weight=None, bias=None, gate=None, activation="silu", eps=1e-5,
                        rms=False, dx=None, dgate=None, dweight=None, dbias=None, workspace=None,
                        stream=None):
    """group_norm_backward.  Returns (dx, dweight, dbias, dgate), the gradients of sum <y, dy> for the
    inputs of :func:`group_norm_forward`, from those alone; None for inputs that are not given.  ``dx``
    may be ``dy`` (in place)."""
    import torch

    p = _problem(torch, x, groups, weight, bias, gate, activation, eps, rms)
    dt, dev = x.dtype, x.device
    if dy is None:
        raise ValueError("the backward needs dy")
    for name, t in (("dy", dy), ("dx", dx), ("dgate", dgate)):
        _dense(t, name, x.shape, dt, dev)
    for name, t, of in (("dweight", dweight, weight), ("dbias", dbias, bias)):
        _dense(t, name, x.shape[-1:], torch.float32, dev)
        if t is not None and of is None:
            raise ValueError(f"{name} without {name[1:]}")
    if dgate is not None and gate is None:
        raise ValueError("dgate without gate")
    with _On(torch, dev, stream) as on:
        on.uses(x, dy, weight, bias, gate, dx, dgate, dweight, dbias)
        dx = on.like(x) if dx is None else dx
        if gate is not None and dgate is None:
            dgate = on.like(x)
        if weight is not None and dweight is None:
            dweight = on.like(weight)
        if bias is not None and dbias is None:
            dbias = on.like(bias)
        ref = ctypes.byref(p)
        need = 0 if dweight is None and dbias is None else lib().group_norm_backward_workspace(ref)
        workspace, size = on.workspace(need, workspace)
        _check(lib().group_norm_backward(
            ref, _ptr(x), _ptr(gate), _ptr(weight), _ptr(bias), _ptr(dy), _ptr(dx), _ptr(dgate), _ptr(dweight),
            _ptr(dbias), _ptr(workspace), size, on.handle), "group_norm_backward")
    return dx, dweight, dbias, dgate
