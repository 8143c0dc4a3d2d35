"""The training step's stored states away from where the forward wrote them: copied, and through autograd's
hooks on saved tensors."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T, HK, HV = 150, 1, 2


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


def inputs(dtype, K, V):
    gen = torch.Generator("cuda").manual_seed(2)
    new = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x = [new(1, T, HK, K), new(1, T, HK, K), new(1, T, HV, V), -new(1, T, HV).abs(), new(1, T, HV).sigmoid()]
    return [t.to(dtype) for t in x], new(1, T, HV, V).to(dtype)


@pytest.mark.parametrize("dtype,name", [(torch.bfloat16, "bf16"), (torch.float32, "f32")])
@pytest.mark.parametrize("K,V", [(64, 128), (128, 64)])
def test_a_copy_of_the_dense_form(rnn, dtype, name, K, V):
    x, d_o = inputs(dtype, K, V)
    o, s, ck, u = rnn.gated_delta_forward_train(*x, normalize=True)
    want = rnn.gated_delta_backward(*x, d_o, ck, u, normalize=True)
    store = torch.empty(rnn.gated_delta_chunks(T), HV, rnn.gated_delta_ckpt_size(V, K, dtype=name), dtype=dtype,
                        device="cuda")
    o2, s2, ck2, u2 = rnn.gated_delta_forward_train(*x, normalize=True, s_ckpt=store)
    assert ck2 is store and torch.equal(o, o2) and torch.equal(s, s2) and torch.equal(u, u2)
    away = store.cpu()
    store.fill_(float("nan"))
    got = rnn.gated_delta_backward(*x, d_o, away.cuda(), u, normalize=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_hooks_on_saved_tensors(rnn):
    x, d_o = inputs(torch.bfloat16, 64, 64)

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *x):
            store = torch.empty(rnn.gated_delta_chunks(T), HV, rnn.gated_delta_ckpt_size(64, 64), dtype=torch.bfloat16,
                                device="cuda")
            o, _, _, u = rnn.gated_delta_forward_train(*x, normalize=True, s_ckpt=store)
            ctx.save_for_backward(*x, store, u)
            return o

        @staticmethod
        def backward(ctx, d_o):
            *x, store, u = ctx.saved_tensors
            return rnn.gated_delta_backward(*x, d_o.contiguous(), store, u, normalize=True)[:5]

    def grads():
        leaves = [t.clone().requires_grad_() for t in x]
        o = Layer.apply(*leaves)
        return torch.autograd.grad(o, leaves, d_o)

    want = grads()
    with torch.autograd.graph.save_on_cpu():
        got = grads()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _, _, ck, u = rnn.gated_delta_forward_train(*x, normalize=True)
    plain = rnn.gated_delta_backward(*x, d_o, ck, u, normalize=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, want))
