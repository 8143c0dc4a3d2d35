"""Calls on a given stream while the current one is still busy with memory that the host has freed:
a kernel that waits keeps the current stream's work behind it for a while."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DELAY = 20_000_000  # ticks of the GPU: 10 ms or more


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


def gated_inputs(seed, T=300, Hk=2, Hv=4, K=128, V=128):
    g = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    x = [new(1, T, Hk, K), new(1, T, Hk, K), new(1, T, Hv, V), -new(1, T, Hv).abs(), new(1, T, Hv).sigmoid()]
    return [t.bfloat16() for t in x]


def tensors(out):
    return [t for t in out if t is not None] if isinstance(out, tuple) else [out]


def gated_calls(rnn):
    x = gated_inputs(1)
    T, Hk, Hv, K, V = 300, 2, 4, 128, 128
    o, s, ck, u = rnn.gated_delta_forward_train(*x, normalize=True)
    d_o = torch.randn_like(o)
    states = torch.randn(1, 4, Hv, V, K, device="cuda").expand(4, -1, -1, -1, -1).contiguous()
    left = list(states)  # each decode call updates one
    one = [t[0, :4].contiguous() for t in x]
    fwd = rnn.gated_delta_forward_workspace_bytes(T, Hk, Hv, K, V)
    bwd = rnn.gated_delta_backward_workspace_bytes(T, Hk, Hv, K, V)
    return {
        "forward": (lambda **k: rnn.gated_delta_forward(*x, normalize=True, **k), fwd),
        "train": (lambda **k: rnn.gated_delta_forward_train(*x, normalize=True, **k), fwd),
        "backward": (lambda **k: rnn.gated_delta_backward(*x, d_o, ck, u, normalize=True, **k), bwd),
        "decode": (lambda **k: rnn.gated_delta_decode(*one, left.pop(), normalize=True, **k), 0),
    }


def check_busy_memory(call, work):
    """`call` on another stream right after the current one's temporaries, of the sizes of its results and its
    workspace, have been freed on the host with their kernels still to run."""
    want = tensors(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        used = [torch.empty_like(t) for t in want] + [torch.empty(work, dtype=torch.uint8, device="cuda")]
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(DELAY)
        for t in used:
            t.fill_(7)
        del used, t
        got = tensors(call(stream=side))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def check_results_freed(call):
    """Results that the current stream still has to read when the host frees them stay until then, whatever the
    given stream is asked for meanwhile."""
    want = tensors(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        got = tensors(call(stream=side))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(DELAY)
        copies = [t.clone() for t in got]
        with torch.cuda.stream(side):
            shapes = [(t.shape, t.dtype) for t in got]
            del got
            for shape, dtype in shapes:
                torch.empty(shape, dtype=dtype, device="cuda").fill_(7)
        torch.cuda.synchronize()
        for a, b in zip(copies, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["forward", "train", "backward", "decode"])
def test_gated_delta_leaves_busy_memory_alone(rnn, name):
    call, work = gated_calls(rnn)[name]
    check_busy_memory(call, work)


@pytest.mark.parametrize("name", ["forward", "train", "backward", "decode"])
def test_gated_delta_results_may_be_freed_at_any_time(rnn, name):
    check_results_freed(gated_calls(rnn)[name][0])


def test_gated_delta_inputs_may_be_freed_at_once(rnn):
    """Inputs that the host frees behind the call are not overwritten by the current stream before the given
    stream, which is still waiting, has read them."""
    x = gated_inputs(2)
    want = rnn.gated_delta_forward(*x, normalize=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    y = [t.clone() for t in x]
    side.wait_stream(torch.cuda.current_stream())
    o, s = rnn.gated_delta_forward(*y, normalize=True, stream=side)
    shapes = [t.shape for t in y]
    del y
    for shape in shapes:
        torch.empty(shape, dtype=torch.bfloat16, device="cuda").fill_(7)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(s, want[1])


def wkv_calls(rnn):
    B, T, H, N = 2, 400, 3, 64
    g = torch.Generator("cuda").manual_seed(3)
    new = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    kappa = torch.nn.functional.normalize(new(B, T, H, N), dim=-1)
    x = [t.bfloat16() for t in (new(B, T, H, N), new(B, T, H, N).sigmoid() * 0.5 + 0.5, new(B, T, H, N), new(B, T, H, N),
                                kappa, new(B, T, H, N).sigmoid())]
    r, w, k, v, kappa, a = x
    y, s, ck = rnn.forward_train(*x)
    dy = torch.randn_like(y)
    key = [torch.ones(H * N, device="cuda"), torch.ones(H * N, device="cuda")]
    states = torch.randn(1, B, H, N, N, device="cuda").expand(4, -1, -1, -1, -1).contiguous()
    left = list(states)
    one = [t[:, 0].contiguous() for t in x]
    fwd, bwd = rnn.forward_workspace_bytes(B, T, H), rnn.backward_workspace_bytes(B, T, H)
    return {
        "forward": (lambda **o: rnn.forward(*x, **o), fwd),
        "bidir": (lambda **o: rnn.forward_bidir(*x, **o), rnn.forward_bidir_workspace_bytes(B, T, H)),
        "fused": (lambda **o: rnn.forward_fused(r, w, k, v, a, *key, **o), fwd),
        "train": (lambda **o: rnn.forward_train(*x, **o), fwd),
        "backward": (lambda **o: rnn.backward(*x, dy, ck, **o), bwd),
        "decode": (lambda **o: rnn.decode(*one, left.pop(), **o), 0),
    }


WKV = ["forward", "bidir", "fused", "train", "backward", "decode"]


@pytest.mark.parametrize("name", WKV)
def test_wkv_leaves_busy_memory_alone(rnn, name):
    call, work = wkv_calls(rnn)[name]
    check_busy_memory(call, work)


@pytest.mark.parametrize("name", WKV)
def test_wkv_results_may_be_freed_at_any_time(rnn, name):
    check_results_freed(wkv_calls(rnn)[name][0])
