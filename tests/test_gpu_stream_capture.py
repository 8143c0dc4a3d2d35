"""A captured call on a given stream that the capture has forked to, replayed with eager calls in between."""
import pytest

from tests.test_gpu_stream_memory import gated_inputs, rnn  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_gated_delta_on_a_forked_stream(rnn):  # noqa: F811
    x = gated_inputs(5)
    d_o = torch.randn(1, 300, 4, 128, device="cuda").bfloat16()
    side = torch.cuda.Stream()

    def step(stream):
        o, s, ck, u = rnn.gated_delta_forward_train(*x, normalize=True, stream=stream)
        return [o, s, *rnn.gated_delta_backward(*x, d_o, ck, u, normalize=True, stream=stream)]

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
