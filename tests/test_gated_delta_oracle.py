"""The float64 gated delta rule: closed forms, invariants, and its gradients against
central differences."""
import numpy as np
import pytest

from oracle import gated_delta as gd
import oracle


def draw(T, Hk, Hv, K, V, seed):
    r = np.random.default_rng(seed)
    return (r.normal(size=(T, Hk, K)), r.normal(size=(T, Hk, K)), r.normal(size=(T, Hv, V)),
            -np.abs(r.normal(size=(T, Hv))), 1 / (1 + np.exp(-r.normal(size=(T, Hv)))),
            r.normal(size=(Hv, V, K)))


def test_single_token_closed_form():
    q, k, v, g, beta, s0 = draw(1, 1, 1, 3, 2, 1)
    o, S, _ = gd.forward(q, k, v, g, beta, s0, scale=0.5)
    a, b, kt = np.exp(g[0, 0]), beta[0, 0], k[0, 0]
    want = a * s0[0] @ (np.eye(3) - b * np.outer(kt, kt)) + b * np.outer(v[0, 0], kt)
    np.testing.assert_allclose(S[0], want, rtol=1e-13)
    np.testing.assert_allclose(o[0, 0], 0.5 * want @ q[0, 0], rtol=1e-13)


def test_split_sequences_agree():
    q, k, v, g, beta, s0 = draw(9, 2, 4, 5, 3, 2)
    o, S, _ = gd.forward(q, k, v, g, beta, s0, normalize=True)
    o1, S1, _ = gd.forward(q[:4], k[:4], v[:4], g[:4], beta[:4], s0, normalize=True)
    o2, S2, _ = gd.forward(q[4:], k[4:], v[4:], g[4:], beta[4:], S1, normalize=True)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, rtol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12)


def test_full_write_strength_replaces_what_the_key_recalls():
    q, k, v, g, beta, s0 = draw(6, 1, 1, 4, 4, 3)
    k = k / np.linalg.norm(k, axis=-1, keepdims=True)
    o, S, _ = gd.forward(q, k, v, 0 * g, 1 + 0 * beta, s0)
    np.testing.assert_allclose(S[0] @ k[-1, 0], v[-1, 0], rtol=1e-12)


def test_it_is_the_wkv7_update_with_a_scalar_decay():
    """w = exp(g), kappa = k, a = beta exp(g), and the written key beta k give the same state."""
    T, H, N = 7, 2, 64
    q, k, v, g, beta, s0 = draw(T, H, H, N, N, 4)
    k = k / np.linalg.norm(k, axis=-1, keepdims=True)
    one = np.ones((T, H, N))
    w, b = np.exp(g)[..., None] * one, beta[..., None]
    y, S = oracle.forward(*(x[None] for x in (q, w, b * k, v, k, w * b * one)), s0=s0[None])
    o, S2, _ = gd.forward(q, k, v, g, beta, s0, scale=1.0)
    np.testing.assert_allclose(y[0], o, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(S[0], S2, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("normalize", [False, True])
def test_gradients_against_differences(normalize):
    q, k, v, g, beta, s0 = draw(4, 1, 2, 3, 2, 5)
    r = np.random.default_rng(6)
    d_o, ds = r.normal(size=(4, 2, 2)), r.normal(size=(2, 2, 3))
    x = [q, k, v, g, beta, s0]
    grads = gd.backward(q, k, v, g, beta, d_o, ds, s0, normalize=normalize)

    def loss(y):
        o, S, _ = gd.forward(*y, normalize=normalize)
        return (o * d_o).sum() + (S * ds).sum()

    for i, d in enumerate(grads):
        for at in np.ndindex(*x[i].shape):
            lo, hi = [a.copy() for a in x], [a.copy() for a in x]
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            # central differences: (1e-5)^2 of the third derivative, and 1e-16 / 1e-5 of the loss
            assert abs((loss(hi) - loss(lo)) / 2e-5 - d[at]) < 1e-7 * max(1, np.abs(d).max()), (i, at)


def test_moves_read_the_old_pool():
    pool = np.arange(2 * 4 * 3.0).reshape(2, 4, 3)
    new = gd.move(pool, [1, 0, -1, 2, 9, 0], [0, 1, 2, 3, 3, -1])
    np.testing.assert_array_equal(new[:, 0], pool[:, 1])
    np.testing.assert_array_equal(new[:, 1], pool[:, 0])
    assert not new[:, 2].any()
    np.testing.assert_array_equal(new[:, 3], pool[:, 2])
    np.testing.assert_array_equal(gd.move(pool, [0, 1], [3, 3])[:, 3], pool[:, 1])
