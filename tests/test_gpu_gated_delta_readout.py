"""How exact bf16 readouts are: o and P are rounded to bf16, everything else that enters o has 16 bits
of significand.

A rounding of normally distributed numbers is off by 1.66e-3 of them in the mean (2^-8 / sqrt(3) of the
lower end of a binade).  P U is not larger than o itself where the entry state and the chunk's own tokens
add up as independent parts do, so two such roundings give at most sqrt(2) * 1.66e-3 = 2.35e-3, and the 16 bits
add 2^-17 or so of the parts.  (A third one, of U, would make it 2.6e-3.)"""
import numpy as np
import pytest

from oracle import gated_delta as gd

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


def test_the_mean_rounding():
    x = torch.from_numpy(np.random.default_rng(0).normal(size=1 << 20))
    assert float((x.bfloat16().double() - x).norm() / x.norm()) <= 1.67e-3


# the workgroups of four and eight waves, both key widths, and (one long sequence) segments
@pytest.mark.parametrize("n,T,Hk,Hv,K,V", [(2, 500, 2, 4, 128, 128), (2, 500, 2, 4, 64, 64), (1, 1100, 1, 2, 128, 128),
                                           (1, 1100, 1, 2, 64, 128)])
def test_readouts(rnn, n, T, Hk, Hv, K, V):
    r = np.random.default_rng(T + K)
    x = [r.normal(size=(n, T, Hk, K)), r.normal(size=(n, T, Hk, K)), r.normal(size=(n, T, Hv, V)),
         -np.exp(r.uniform(np.log(0.01), 0, size=Hv)) * np.log1p(np.exp(r.normal(size=(n, T, Hv)))),
         1 / (1 + np.exp(-r.normal(size=(n, T, Hv))))]
    x = [torch.from_numpy(a).bfloat16().cuda() for a in x]
    o, _ = rnn.gated_delta_forward(*x, normalize=True)
    ot = rnn.gated_delta_forward_train(*x, normalize=True)[0]
    assert torch.equal(o, ot)
    for i in range(n):
        want = gd.forward(*(a[i].double().cpu().numpy() for a in x), normalize=True)[0]
        off = np.linalg.norm(o[i].double().cpu().numpy() - want) / np.linalg.norm(want)
        assert off <= 2.4e-3, off
