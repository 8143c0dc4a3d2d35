"""Linear attention and the group norm on a given stream: while the current one is still busy with memory that
the host has freed, with results and inputs freed at once, and captured on a stream that the capture forked to."""
import pytest

from tests.test_gpu_stream_memory import DELAY, check_busy_memory, check_results_freed, rnn  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

Hk, Hv, K, V = 2, 4, 128, 128
NAMES = ["forward", "backward", "decode", "norm", "norm_backward"]


def inputs(seed, T):
    g = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()  # noqa: E731
    return [new(1, T, Hk, K), new(1, T, Hk, K), new(1, T, Hv, V), -torch.rand(Hv, device="cuda", generator=g)], \
        new(1, T, Hv, V), torch.randn(Hv * V, device="cuda", generator=g)


def calls(rnn, T):  # noqa: F811
    """Each with the bytes of its workspace."""
    x, d_o, weight = inputs(1, T)
    one = [t[0, :4].contiguous() for t in x[:3]]
    left = list(torch.randn(1, 4, Hv, V, K, device="cuda").expand(4, -1, -1, -1, -1).contiguous())
    rows = d_o.view(T, Hv * V)
    y = x[2].view(T, Hv * V)
    norm = dict(weight=weight, bias=weight, gate=y)
    return {
        "forward": (lambda **k: rnn.linear_attention_forward(*x, **k),
                    rnn.linear_attention_forward_workspace_bytes(T, Hk, Hv, K, V)),
        "backward": (lambda **k: rnn.linear_attention_backward(*x, d_o, **k),
                     rnn.linear_attention_backward_workspace_bytes(T, Hk, Hv, K, V)),
        "decode": (lambda **k: rnn.linear_attention_decode(*one, x[3], left.pop(), **k), 0),
        "norm": (lambda **k: rnn.group_norm_forward(rows, Hv, **norm, **k), 0),
        "norm_backward": (lambda **k: rnn.group_norm_backward(y, Hv, rows, **norm, **k),
                          rnn.group_norm_backward_workspace_bytes(T, Hv, V)),
    }


@pytest.mark.parametrize("T", [300, 700])  # whole, and in segments
@pytest.mark.parametrize("name", NAMES)
def test_busy_memory_is_left_alone(rnn, name, T):  # noqa: F811
    check_busy_memory(*calls(rnn, T)[name])


@pytest.mark.parametrize("name", NAMES)
def test_results_may_be_freed_at_any_time(rnn, name):  # noqa: F811
    check_results_freed(calls(rnn, 300)[name][0])


def test_inputs_may_be_freed_at_once(rnn):  # noqa: F811
    """Inputs that the host frees behind the call are not overwritten by the current stream before the given
    stream, which is still waiting, has read them."""
    x, d_o, weight = inputs(2, 300)

    def step(x, d_o, weight, stream=None):
        return [*rnn.linear_attention_forward(*x, stream=stream), *rnn.linear_attention_backward(*x, d_o, stream=stream),
                rnn.group_norm_forward(d_o.view(300, Hv * V), Hv, weight=weight, stream=stream)]

    want = step(x, d_o, weight)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    copies = [t.clone() for t in (*x, d_o, weight)]
    side.wait_stream(torch.cuda.current_stream())
    got = step(copies[:4], copies[4], copies[5], side)
    shapes = [(t.shape, t.dtype) for t in copies]
    del copies
    for shape, dtype in shapes:
        torch.empty(shape, dtype=dtype, device="cuda").fill_(7)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [300, 700])
def test_captured_on_a_forked_stream(rnn, T):  # noqa: F811
    x, d_o, weight = inputs(3, T)
    side = torch.cuda.Stream()

    def step(stream):
        o, s = rnn.linear_attention_forward(*x, stream=stream)
        flat = [t.view(T, Hv * V) for t in (o, x[2], d_o)]
        y = rnn.group_norm_forward(flat[0], Hv, weight=weight, gate=flat[1], stream=stream)
        dx, dw, _, dgate = rnn.group_norm_backward(flat[0], Hv, flat[2], weight=weight, gate=flat[1], stream=stream)
        return [o, s, y, dx, dw, dgate, *rnn.linear_attention_backward(*x, dx.view(1, T, Hv, V), stream=stream)]

    want = step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = step(side)
        main.wait_stream(side)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        again = step(None)  # eager work while the replay runs
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(c, b)
