"""Plain float64 implementation of the group norm with an activation or gate, and of its gradients
(numpy): each row [C] by itself, in groups of neighbouring channels.

    u = (x - mean) / sqrt(var + eps)  (rms: x / sqrt(mean(x^2) + eps));  n = u weight + bias
    y = n act(gate) with a gate, act(n) without one
"""
from __future__ import annotations

import numpy as np


def _act(z, name):
    """The activation and its derivative."""
    if name == "none":
        return z, np.ones_like(z)
    s = 1 / (1 + np.exp(-z))
    return (s, s * (1 - s)) if name == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def _parts(x, groups, weight, bias, eps, rms):
    rows, C = x.shape
    g = x.reshape(rows, groups, C // groups)
    d = g if rms else g - g.mean(-1, keepdims=True)
    inv = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    unit = (d * inv).reshape(rows, C)
    return unit, inv, unit * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)


def forward(x, groups, *, weight=None, bias=None, gate=None, activation="silu", eps=1e-5, rms=False):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        _, _, n = _parts(x, groups, weight, bias, eps, rms)
        return _act(n, activation)[0] if gate is None else n * _act(np.asarray(gate, np.float64), activation)[0]


def backward(x, groups, dy, *, weight=None, bias=None, gate=None, activation="silu", eps=1e-5, rms=False):
    """(dx, dweight, dbias, dgate) of sum <y, dy>; dgate None without a gate."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    rows, C = x.shape
    with np.errstate(over="ignore"):
        unit, inv, n = _parts(x, groups, weight, bias, eps, rms)
        if gate is None:
            dn, dgate = dy * _act(n, activation)[1], None
        else:
            a, slope = _act(np.asarray(gate, np.float64), activation)
            dn, dgate = dy * a, dy * n * slope
    du = (dn * (1.0 if weight is None else weight)).reshape(rows, groups, -1)
    u = unit.reshape(du.shape)
    dx = du - u * (u * du).mean(-1, keepdims=True)
    if not rms:
        dx = dx - du.mean(-1, keepdims=True)
    return (inv * dx).reshape(rows, C), (dn * unit).sum(0), dn.sum(0), dgate
