"""The decay's gradient from stored states that have few significant bits (they came from float16, or are
halfway between two bf16 numbers), where rounding goes to even.

With nothing written (beta = 0) and nothing read (d_o = 0), dg of every token is the whole decay times
<S0, dS_T>.  A stored state is off by at most 2^-12 of each element, a product by 2^-11 (1 + 2^-13), the
sum by that of the sum of the products' sizes; float32 sums add 2^-24 for each of the at most 2^15 terms
one after the other, 2^-9 at the very worst and 2^-17 for roundings of either sign, which the factor
1.05 holds; the result is rounded to bf16, 2^-8."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


def decay_gradient(rnn, s0, ds, T):
    """dg [B, T] of a bf16 training step that neither writes nor reads, and the decay of all tokens."""
    B, _, V, K = s0.shape
    g = torch.full((B, T, 1), -1.0 / 64, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(B, T, 1, K, device="cuda").bfloat16(), torch.randn(B, T, 1, V, device="cuda").bfloat16()
    beta = torch.zeros_like(g)
    _, _, ck, u = rnn.gated_delta_forward_train(x[0], x[0], x[1], g, beta, s0=s0, normalize=True)
    dg = rnn.gated_delta_backward(x[0], x[0], x[1], g, beta, torch.zeros_like(x[1]), ck, u, ds_T=ds,
                                  normalize=True)[3]
    return dg.double().cpu().numpy()[..., 0], np.exp(-T / 64)


def check(rnn, s0, ds, T):
    dg, c = decay_gradient(rnn, s0, ds, T)
    terms = (s0.double() * ds.double()).cpu().numpy().reshape(len(s0), -1)
    want, size = c * terms.sum(1), c * np.abs(terms).sum(1)
    worst = np.max((np.abs(dg - want[:, None]) - 2.0 ** -8 * np.abs(want[:, None])) / size[:, None])
    assert worst <= 1.05 * 2.0 ** -11


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 64])
@pytest.mark.parametrize("up", [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 257.0])
def test_states_halfway_between_two_bf16_numbers(rnn, K, V, T, up):
    """Half of the elements lie halfway, half are bf16 numbers of the other sign, so that the sum is about the
    distance between them: 2^-8 of the terms, where the bound is 2^-11."""
    s0 = torch.full((2, 1, V, K), float(up), device="cuda")
    s0[..., ::2] = -float(np.floor(up))
    check(rnn, s0, torch.ones_like(s0), T)
    check(rnn, torch.ones_like(s0), s0, T)  # the cotangent is kept the same way


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_states_that_came_from_float16(rnn, K, V):
    """As for any float32 states: of V K terms of either sign, the errors are of either sign too."""
    gen = torch.Generator("cuda").manual_seed(1)
    s0, ds = (torch.randn(128, 1, V, K, device="cuda", generator=gen).half().float() for _ in range(2))
    dg, c = decay_gradient(rnn, s0, ds, 1)
    terms = (s0.double() * ds.double()).cpu().numpy().reshape(len(s0), -1)
    want, size = c * terms.sum(1), c * np.sqrt((terms ** 2).sum(1))
    # uniform errors of up to 2^-12 in each factor: 2^-11 / sqrt(6) of the root sum of squares, six times that
    worst = np.max((np.abs(dg[:, 0] - want) - 2.0 ** -8 * np.abs(want)) / size)
    assert worst <= 2.0 ** -9.7


def test_the_smallest_states(rnn):
    """Elements below bf16's smallest normal number, of which the one with the bits 0x8000 lies halfway between
    0 and the next; zeros; both signs."""
    bits = torch.tensor([0x8000, 0x18000, 0x7fff, 0x8001, 1, 0, 0x7fffff, 0x800000], dtype=torch.int32)
    tiny = torch.cat([bits, bits | -(1 << 31)]).view(torch.float32).cuda()
    s0 = tiny.repeat(64 * 64 // 16).view(1, 1, 64, 64).clone()
    s0[0, 0, 5] = 3.0
    ds = torch.ones_like(s0)
    check(rnn, s0, ds, 1)
    check(rnn, ds, s0, 1)
