"""Plain float64 implementation of the gated delta rule, token by token, and of its
gradients; and of the state moves.  numpy only, one (sequence, value head) at a time:

    Sd = exp(g_t) S;  e_t = v_t - Sd k_t;  S = Sd + beta_t e_t k_t^T;  o_t = scale S q_t

with S [V, K], value head h reading key head h // (Hv // Hk), and q, k divided by
sqrt(sum of squares + 1e-6) first where ``normalize`` is set.  It shares no code and no
chunking with the GPU path.
"""
from __future__ import annotations

import numpy as np

NORM_EPS = 1e-6


def _unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + NORM_EPS)


def forward(q, k, v, g, beta, s0=None, *, scale=None, normalize=False):
    """One sequence: q, k [T,Hk,K], v [T,Hv,V], g, beta [T,Hv], s0 [Hv,V,K].
    Returns (o [T,Hv,V], S [Hv,V,K], trace) with the states before each token."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    T, Hk, K = k.shape
    Hv, V = v.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    if normalize:
        q, k = _unit(q), _unit(k)
    S = np.zeros((Hv, V, K)) if s0 is None else np.array(s0, np.float64)
    o = np.zeros((T, Hv, V))
    trace = []
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            trace.append(S)
            new = np.empty_like(S)
            for h in range(Hv):
                kt, qt = k[t, h // (Hv // Hk)], q[t, h // (Hv // Hk)]
                Sd = np.exp(g[t, h]) * S[h]
                e = v[t, h] - Sd @ kt
                new[h] = Sd + beta[t, h] * np.outer(e, kt)
                o[t, h] = scale * (new[h] @ qt)
            S = new
    return o, S, trace


def backward(q, k, v, g, beta, d_o, ds_T=None, s0=None, *, scale=None, normalize=False):
    """Gradients (dq, dk, dv, dg, dbeta, ds0) of sum <o, d_o> + <S_T, ds_T>, by the chain rule
    applied to one token after the other, last to first."""
    raw_q, raw_k, v, g, beta, d_o = (np.asarray(x, np.float64) for x in (q, k, v, g, beta, d_o))
    T, Hk, K = raw_k.shape
    Hv, V = v.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    q, k = (_unit(raw_q), _unit(raw_k)) if normalize else (raw_q, raw_k)
    _, S_T, trace = forward(raw_q, raw_k, v, g, beta, s0, scale=scale, normalize=normalize)
    after = trace[1:] + [S_T]
    D = np.zeros((Hv, V, K)) if ds_T is None else np.array(ds_T, np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        for h in range(Hv):
            j = h // (Hv // Hk)
            kt, qt, a = k[t, j], q[t, j], np.exp(g[t, h])
            Sd = a * trace[t][h]
            e = v[t, h] - Sd @ kt
            D[h] += scale * np.outer(d_o[t, h], qt)
            dq[t, j] += scale * (after[t][h].T @ d_o[t, h])
            db[t, h] = e @ D[h] @ kt
            dk[t, j] += beta[t, h] * (D[h].T @ e)
            de = beta[t, h] * (D[h] @ kt)
            dv[t, h] = de
            dk[t, j] -= Sd.T @ de
            dSd = D[h] - np.outer(de, kt)
            dg[t, h] = (dSd * Sd).sum()
            D[h] = a * dSd
    if normalize:
        def through(d, x):
            r = np.sqrt((x * x).sum(-1, keepdims=True) + NORM_EPS)
            return d / r - x * (x * d).sum(-1, keepdims=True) / r ** 3
        dq, dk = through(dq, raw_q), through(dk, raw_k)
    return dq, dk, dv, dg, db, D


def move(pool, src, dst):
    """pool [layers, slots, ...] after the moves: every pair reads the old pool; -1 writes zeros;
    pairs out of range are left out; the last of several pairs with one target counts."""
    new = np.array(pool)
    slots = new.shape[1]
    for s, d in zip(src, dst):
        if 0 <= d < slots and -1 <= s < slots:
            new[:, d] = pool[:, s] if s >= 0 else 0
    return new
