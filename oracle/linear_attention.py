"""Plain float64 implementation of linear attention with a decay for each head, token by token,
and of its gradients.  numpy only, one sequence at a time:

    S = exp(g_h) S + v_t k_t^T;  o_t = scale S q_t

with S [V, K], value head h reading key head h // (Hv // Hk).  It shares no code and no chunking
with the GPU path.
"""
from __future__ import annotations

import numpy as np


def _inputs(*xs):
    return [np.asarray(x, np.float64) for x in xs]


def forward(q, k, v, g, s0=None, *, scale=None):
    """q, k [T,Hk,K], v [T,Hv,V], g [Hv], s0 [Hv,V,K].  Returns (o [T,Hv,V], S [Hv,V,K], trace)
    with the states before each token."""
    q, k, v, g = _inputs(q, k, v, g)
    T, Hk, K = k.shape
    Hv, V = v.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    S = np.zeros((Hv, V, K)) if s0 is None else np.array(s0, np.float64)
    a = np.exp(g)[:, None, None]
    rep = Hv // Hk
    o, trace = np.zeros((T, Hv, V)), []
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            trace.append(S)
            kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
            S = a * S + v[t][:, :, None] * kt[:, None, :]
            o[t] = scale * (S * qt[:, None, :]).sum(-1)
    return o, S, trace


def backward(q, k, v, g, d_o, ds_T=None, s0=None, *, scale=None):
    """Gradients (dq, dk, dv, dg, ds0) of sum <o, d_o> + <S_T, ds_T>, by the chain rule applied to
    one token after the other, last to first."""
    q, k, v, g, d_o = _inputs(q, k, v, g, d_o)
    T, Hk, K = k.shape
    Hv, V = v.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    _, S_T, trace = forward(q, k, v, g, s0, scale=scale)
    after = trace[1:] + [S_T]
    D = np.zeros((Hv, V, K)) if ds_T is None else np.array(ds_T, np.float64)
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(g)
    a = np.exp(g)[:, None, None]
    rep = Hv // Hk
    for t in range(T - 1, -1, -1):
        kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
        dq[t] = scale * (after[t] * d_o[t][:, :, None]).sum(1).reshape(Hk, rep, K).sum(1)
        D = D + scale * d_o[t][:, :, None] * qt[:, None, :]
        dk[t] = (D * v[t][:, :, None]).sum(1).reshape(Hk, rep, K).sum(1)
        dv[t] = (D * kt[:, None, :]).sum(-1)
        D = a * D
        dg += (D * trace[t]).sum((1, 2))
    return dq, dk, dv, dg, D
