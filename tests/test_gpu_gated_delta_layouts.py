"""The gated delta rule at three quarters of the largest V and at four to six value heads a key head,
against float64: prefill, single tokens and training, few chunks and many."""
import numpy as np
import pytest

from oracle import gated_delta as gd
from tests.test_gpu_gated_delta import DT, NAMES, close, close_state, f64, inputs, rows, states

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# (dtype, K, V, Hk, Hv)
LAYOUTS = [("bf16", 64, 192, 1, 2), ("bf16", 128, 192, 2, 2), ("f32", 64, 192, 1, 1), ("f32", 128, 192, 1, 2),
           ("bf16", 64, 64, 1, 4), ("bf16", 128, 128, 1, 4), ("bf16", 64, 64, 1, 5), ("f32", 64, 64, 2, 12),
           ("bf16", 64, 256, 1, 1), ("f32", 64, 256, 1, 4)]


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(12)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("T", [1, 70, 129])
def test_training_step(rnn, layout, T):
    dtype, K, V, Hk, Hv = layout
    x = inputs(T, Hk, Hv, K, V, dtype, 200 + T, slow=True)
    s0, ds = states(1, Hv, V, K, 1), states(1, Hv, V, K, 2)
    d_o = torch.from_numpy(np.random.default_rng(9).normal(size=(1, T, Hv, V))).to(DT[dtype]).cuda()
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, normalize=True)
    plain = rnn.gated_delta_forward(*x.values(), s0=s0, normalize=True)
    assert torch.equal(o, plain[0]) and torch.equal(s, plain[1])
    want, S, trace = gd.forward(*rows(x, 0, 0, T), f64(s0[0]), normalize=True)
    close(o[0], want, dtype, "o")
    close_state(s[0], S, dtype)
    for c in range(ck.shape[0]):
        close(ck[c], trace[64 * c], dtype, f"state {c}")
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, normalize=True)
    ref = gd.backward(*rows(x, 0, 0, T), f64(d_o[0]), f64(ds[0]), f64(s0[0]), normalize=True)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
        close(a[0], b, dtype, n)
    close_state(grads[5][0], ref[5], dtype, "ds0")


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_single_tokens(rnn, layout):
    dtype, K, V, Hk, Hv = layout
    B, steps = 3, 2
    x = inputs(B * steps, Hk, Hv, K, V, dtype, 210, B=B)
    pool = states(B, Hv, V, K, 3)
    old = pool.clone()
    os = [rnn.gated_delta_decode(*(a[:, t].contiguous() for a in x.values()), pool, normalize=True)
          for t in range(steps)]
    for b in range(B):
        want, S, _ = gd.forward(*rows(x, b, 0, steps), f64(old[b]), normalize=True)
        close(torch.stack([o[b] for o in os]), want, dtype, "o")
        close_state(pool[b], S, "f32")


@pytest.mark.parametrize("layout", [LAYOUTS[1], LAYOUTS[3], LAYOUTS[5], LAYOUTS[6], LAYOUTS[7]], ids=str)
def test_many_sequences(rnn, layout):
    """More chunks than CUs: one workgroup prepares all value heads of a key head, two at a time."""
    dtype, K, V, Hk, Hv = layout
    n = 300
    r = np.random.default_rng(7)
    lens = r.integers(0, 100, n)
    cu = np.cumsum([0, *lens])
    x = inputs(int(cu[-1]), Hk, Hv, K, V, dtype, 220)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s0, ds = states(n, Hv, V, K, 1), states(n, Hv, V, K, 2)
    d_o = torch.randn(1, int(cu[-1]), Hv, V, device="cuda").to(DT[dtype])
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, cu_seqlens=cut, normalize=True)
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, cu_seqlens=cut, normalize=True)
    for i in range(0, n, 25):
        a, b = cu[i], cu[i + 1]
        want, S, _ = gd.forward(*rows(x, 0, a, b), f64(s0[i]), normalize=True)
        ref = gd.backward(*rows(x, 0, a, b), f64(d_o[0, a:b]), f64(ds[i]), f64(s0[i]), normalize=True)
        close(o[0, a:b], want, dtype, f"o of sequence {i}")
        close_state(s[i], S, dtype)
        for name, got, w in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
            close(got[0, a:b], w, dtype, f"{name} of sequence {i}")
        close_state(grads[5][i], ref[5], dtype, f"ds0 of sequence {i}")


@pytest.mark.parametrize("layout", [LAYOUTS[1], LAYOUTS[2], LAYOUTS[4]], ids=str)
def test_segments(rnn, layout):
    dtype, K, V, Hk, Hv = layout
    T = 1300
    x = inputs(T, Hk, Hv, K, V, dtype, 230, slow=True)
    s0 = states(1, Hv, V, K, 8)
    need = rnn.gated_delta_forward_workspace_bytes
    assert need(T, Hk, Hv, K, V, dtype=dtype) > need(64, 1, 1, K, V, dtype=dtype) * Hv * ((T + 63) // 64)
    o, s = rnn.gated_delta_forward(*x.values(), s0=s0, normalize=True)
    want, S, _ = gd.forward(*rows(x, 0, 0, T), f64(s0[0]), normalize=True)
    close(o[0], want, dtype, "o")
    close_state(s[0], S, dtype)


def test_a_long_prompt_next_to_single_tokens(rnn):
    """A long prompt packed with one-token ones that continue other slots or start from zeros."""
    dtype, K, V, Hk, Hv = "bf16", 64, 64, 1, 2
    lens = [700] + [1] * 20
    cu = np.cumsum([0] + lens)
    x = inputs(int(cu[-1]), Hk, Hv, K, V, dtype, 240, slow=True)
    pool = states(24, Hv, V, K, 4)
    old = pool.clone()
    slots = np.random.default_rng(1).permutation(24)[:21]
    start = np.where(np.arange(21) % 3 == 0, -1, slots)
    t32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    o, _ = rnn.gated_delta_forward(*x.values(), s0=pool, s_out=pool, cu_seqlens=t32(cu), slots=t32(slots),
                                   slots_in=t32(start), normalize=True)
    for i in range(21):
        a, b = cu[i], cu[i + 1]
        s0 = f64(old[slots[i]]) if start[i] >= 0 else None
        want, S, _ = gd.forward(*rows(x, 0, a, b), s0, normalize=True)
        close(o[0, a:b], want, dtype, f"o of sequence {i}")
        close_state(pool[slots[i]], S, dtype)
    assert set(NAMES) == set(x)
