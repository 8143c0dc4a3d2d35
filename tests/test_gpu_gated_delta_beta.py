"""The gradient of the write strength where the state recalls the values well, so that v and S k cancel.

dbeta_t = dR_t . e_t, with e_t the error that the token corrects and dR_t the gradient of beta_t e_t's
right side.  The kernels keep u = beta e and dR in the inputs' type: each factor of a product is off by
half a step of it (bf16: 2^-8, float32: 2^-24), the sum by twice that of the sum of the products'
sizes.  e itself is a float32 result: with bf16 inputs its operands are split into 16 bits of
significand (2^-17), for S k, for what the chunk's earlier tokens wrote and for T's product, with
2^-15 in all, relative to the sizes of the products of v - S k; with float32 inputs 2^-20 holds the
sums of up to 128 + 64 terms of either sign (2^-24 each, sqrt(192) < 2^4).  The result is rounded once."""
import numpy as np
import pytest

from oracle import gated_delta as gd

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
FLOATS = {"f32": 2.0 ** -20, "bf16": 2.0 ** -15}


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).double().numpy()


def recalled(T, Hk, Hv, K, V, dtype, seed, off, beta=None):
    """Inputs of one sequence whose values are what the state recalls, but for `off` of their size."""
    r = np.random.default_rng(seed)
    q, k = (r.normal(size=(T, Hk, K)) for _ in range(2))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    q, k = rounded(q, dtype), rounded(k, dtype)
    g = rounded(-0.01 * r.random((T, Hv)), dtype)
    beta = rounded(1 / (1 + np.exp(-r.normal(size=(T, Hv)))) if beta is None else np.full((T, Hv), beta), dtype)
    s0 = r.normal(size=(Hv, V, K)).astype(np.float32).astype(np.float64)
    v, S = np.empty((T, Hv, V)), s0.copy()
    for t in range(T):
        for h in range(Hv):
            kt = k[t, h // (Hv // Hk)]
            Sd = np.exp(g[t, h]) * S[h]
            v[t, h] = rounded(Sd @ kt + off * r.normal(size=V), dtype)
            S[h] = Sd + beta[t, h] * np.outer(v[t, h] - Sd @ kt, kt)
    return q, k, v, g, beta, s0, rounded(r.normal(size=(T, Hv, V)), dtype), r.normal(size=(Hv, V, K)).astype(np.float32)


def gradient(rnn, x, s0, d_o, ds, dtype):
    y = [torch.from_numpy(a)[None].to(DT[dtype]).cuda() for a in (*x, d_o)]
    s0, ds = torch.from_numpy(s0)[None].float().cuda(), torch.from_numpy(ds)[None].cuda()
    _, _, ck, u = rnn.gated_delta_forward_train(*y[:5], s0=s0)
    return rnn.gated_delta_backward(*y[:5], y[5], ck, u, ds_T=ds)[4][0].double().cpu().numpy()


@pytest.mark.parametrize("layout", [("bf16", 64, 64, 1, 2), ("bf16", 128, 128, 2, 4), ("bf16", 128, 64, 1, 1),
                                    ("f32", 64, 64, 1, 2), ("f32", 128, 128, 1, 2)], ids=str)
@pytest.mark.parametrize("T", [1, 64, 130])
@pytest.mark.parametrize("beta", [None, 2.0 ** -30])
def test_write_strengths_of_recalled_values(rnn, layout, T, beta):
    dtype, K, V, Hk, Hv = layout
    *x, s0, d_o, ds = recalled(T, Hk, Hv, K, V, dtype, T, 2.0 ** -6, beta)
    got = gradient(rnn, x, s0, d_o, ds, dtype)
    q, k, v, g, be = x
    ref = gd.backward(*x, d_o, ds.astype(np.float64), s0)
    dR = ref[2] / be[..., None]
    _, _, trace = gd.forward(*x, s0)
    for t in range(T):
        for h in range(Hv):
            kt = k[t, h // (Hv // Hk)]
            Sd = np.exp(g[t, h]) * trace[t][h]
            e = v[t, h] - Sd @ kt
            d = np.abs(dR[t, h])
            bound = 2.01 * STEP[dtype] * (d * np.abs(e)).sum() + STEP[dtype] * abs(ref[4][t, h]) \
                + FLOATS[dtype] * (d * (np.abs(v[t, h]) + np.abs(Sd) @ np.abs(kt))).sum()
            assert abs(got[t, h] - ref[4][t, h]) <= bound, (t, h, got[t, h], ref[4][t, h], bound)
