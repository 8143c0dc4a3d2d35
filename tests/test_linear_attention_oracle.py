"""The float64 linear attention: closed forms, invariants, and its gradients against central
differences."""
import numpy as np

from oracle import gated_delta as gd
from oracle import linear_attention as la


def draw(T, Hk, Hv, K, V, seed):
    r = np.random.default_rng(seed)
    return (r.normal(size=(T, Hk, K)), r.normal(size=(T, Hk, K)), r.normal(size=(T, Hv, V)),
            -np.abs(r.normal(size=Hv)), r.normal(size=(Hv, V, K)))


def test_all_pairs_closed_form():
    """o_t = scale (a^(t+1) S0 q_t + sum_{j <= t} a^(t-j) (q_t . k_j) v_j), a sum over pairs of tokens."""
    T, Hk, Hv = 7, 2, 4
    q, k, v, g, s0 = draw(T, Hk, Hv, 5, 3, 1)
    o, S, _ = la.forward(q, k, v, g, s0, scale=0.5)
    for h in range(Hv):
        a, j = np.exp(g[h]), h // 2
        for t in range(T):
            want = a ** (t + 1) * s0[h] @ q[t, j] + sum(a ** (t - i) * (q[t, j] @ k[i, j]) * v[i, h]
                                                        for i in range(t + 1))
            np.testing.assert_allclose(o[t, h], 0.5 * want, rtol=1e-12, atol=1e-13)
        want = a ** T * s0[h] + sum(a ** (T - 1 - i) * np.outer(v[i, h], k[i, j]) for i in range(T))
        np.testing.assert_allclose(S[h], want, rtol=1e-12, atol=1e-13)


def test_split_sequences_agree():
    q, k, v, g, s0 = draw(9, 2, 4, 5, 3, 2)
    o, S, _ = la.forward(q, k, v, g, s0)
    o1, S1, _ = la.forward(q[:4], k[:4], v[:4], g, s0)
    o2, S2, _ = la.forward(q[4:], k[4:], v[4:], g, S1)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, rtol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12)


def test_decays_of_one_and_none():
    q, k, v, g, s0 = draw(6, 1, 1, 4, 4, 3)
    _, S, _ = la.forward(q, k, v, 0 * g, s0)
    np.testing.assert_allclose(S[0], s0[0] + np.einsum("tv,tk->vk", v[:, 0], k[:, 0]), rtol=1e-12)
    o, S, _ = la.forward(q, k, v, g - np.inf, s0, scale=1.0)
    np.testing.assert_allclose(S[0], np.outer(v[-1, 0], k[-1, 0]), rtol=1e-15)
    np.testing.assert_allclose(o[:, 0], (q[:, 0] * k[:, 0]).sum(-1)[:, None] * v[:, 0], rtol=1e-12)


def test_orthogonal_keys_leave_the_delta_rule_nothing_to_correct():
    T, K = 4, 4
    q, _, v, g, _ = draw(T, 1, 2, K, 3, 4)
    k = np.eye(K)[:, None, :]
    o, S, _ = la.forward(q, k, v, g)
    o2, S2, _ = gd.forward(q, k, v, np.broadcast_to(g, (T, 2)), np.ones((T, 2)))
    np.testing.assert_allclose(o, o2, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(S, S2, rtol=1e-12, atol=1e-14)


def test_gradients_against_differences():
    q, k, v, g, s0 = draw(4, 1, 2, 3, 2, 5)
    r = np.random.default_rng(6)
    d_o, ds = r.normal(size=(4, 2, 2)), r.normal(size=(2, 2, 3))
    x = [q, k, v, g, s0]
    grads = la.backward(q, k, v, g, d_o, ds, s0)

    def loss(y):
        o, S, _ = la.forward(*y)
        return (o * d_o).sum() + (S * ds).sum()

    for i, d in enumerate(grads):
        for at in np.ndindex(*x[i].shape):
            lo, hi = [a.copy() for a in x], [a.copy() for a in x]
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            # central differences: (1e-5)^2 of the third derivative, and 1e-16 / 1e-5 of the loss
            assert abs((loss(hi) - loss(lo)) / 2e-5 - d[at]) < 1e-7 * max(1, np.abs(d).max()), (i, at)
