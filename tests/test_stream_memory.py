"""Which stream's memory a call with a given stream takes: the given one's, since the current
stream may still be using what was freed on the host.  CPU only, with a stand-in for torch that
notes the stream of each allocation."""
import contextlib
import sys
import types

import pytest

pytest.importorskip("torch")
from linear_rnn_sequence_amd import gated_delta as G  # noqa: E402
from linear_rnn_sequence_amd import wkv as W  # noqa: E402


class Stream:
    def __init__(self, device, handle):
        self.device, self.cuda_stream = device, handle


class Memory:
    def __init__(self, stream):
        self.stream, self.recorded = stream, []

    def record_stream(self, stream):
        self.recorded.append(stream)

    def is_contiguous(self):
        return True


def fake_torch(device, current):
    state = {"current": current}

    @contextlib.contextmanager
    def stream(s):
        before, state["current"] = state["current"], s
        try:
            yield
        finally:
            state["current"] = before

    cuda = types.SimpleNamespace(current_device=lambda: device.index, current_stream=lambda d=None: state["current"],
                                 stream=stream, device=lambda d: contextlib.nullcontext())
    new = lambda *a, **k: Memory(state["current"])  # noqa: E731
    return types.SimpleNamespace(cuda=cuda, empty=new, empty_like=new, uint8=None,
                                 _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: state["current"].cuda_stream))


DEVICE = types.SimpleNamespace(type="cuda", index=0)


def test_gated_delta_memory_belongs_to_the_given_stream():
    mine, side = Stream(DEVICE, 1), Stream(DEVICE, 2)
    torch = fake_torch(DEVICE, mine)
    x = Memory(mine)
    x.shape, x.dtype = (2, 3), None
    with G._On(torch, DEVICE, side) as on:
        out, like, (work, _) = on.empty((4,), None), on.like(x), on.workspace(64, None)
        assert on.handle == 2
    assert out.stream is side and like.stream is side and work.stream is side
    # the results may be read on the caller's stream, and freed there
    assert mine in out.recorded and mine in like.recorded
    assert torch.cuda.current_stream() is mine


def test_gated_delta_inputs_are_held_for_the_given_stream():
    mine, side = Stream(DEVICE, 1), Stream(DEVICE, 2)
    x, y = Memory(mine), Memory(mine)
    with G._On(fake_torch(DEVICE, mine), DEVICE, side) as on:
        on.uses(x, None, y)
    with G._On(fake_torch(DEVICE, mine), DEVICE, None) as on:
        on.uses(y)
    assert x.recorded == [side] and y.recorded == [side]


def test_gated_delta_memory_without_a_given_stream():
    mine = Stream(DEVICE, 1)
    torch = fake_torch(DEVICE, mine)
    with G._On(torch, DEVICE, None) as on:
        out, (work, _) = on.empty((4,), None), on.workspace(64, None)
        assert on.handle == 1
    assert out.stream is mine and work.stream is mine and not out.recorded


def test_gated_delta_refuses_another_devices_stream():
    other = types.SimpleNamespace(type="cuda", index=1)
    with pytest.raises(ValueError, match="stream"):
        G._On(fake_torch(DEVICE, Stream(DEVICE, 1)), DEVICE, Stream(other, 2))


def wkv_forward(monkeypatch, stream):
    """A forward call on stand-ins: the stream of its readout, state and workspace, and its input r."""
    real = pytest.importorskip("torch")
    mine = Stream(DEVICE, 1)
    torch = fake_torch(DEVICE, mine)
    torch.bfloat16, torch.float32 = real.bfloat16, real.float32
    seen = {}

    def call(*args):
        seen["stream"] = args[-1].value
        return 0

    lib = types.SimpleNamespace(rwkv7_wkv_forward=call, rwkv7_wkv_forward_workspace=lambda *a: 64)
    monkeypatch.setitem(sys.modules, "torch", torch)
    monkeypatch.setattr(W, "lib", lambda: lib)
    monkeypatch.setattr(Memory, "data_ptr", lambda self: seen.setdefault(self.stream, []).append(self) or 16, raising=False)
    monkeypatch.setattr(Memory, "numel", lambda self: 64, raising=False)
    monkeypatch.setattr(Memory, "element_size", lambda self: 1, raising=False)
    x = []
    for _ in range(6):
        t = Memory(mine)
        t.shape, t.dtype, t.device = (2, 3, 4, 64), real.bfloat16, DEVICE
        x.append(t)
    y, s = W.forward(*x, stream=stream)
    return seen, mine, x, y, s


def test_wkv_memory_belongs_to_the_given_stream(monkeypatch):
    side = Stream(DEVICE, 2)
    seen, mine, x, y, s = wkv_forward(monkeypatch, side)
    assert seen["stream"] == 2
    assert len(seen[mine]) == 6 and len(seen[side]) == 3  # the inputs; readout, state and workspace
    assert y.recorded == [mine] and s.recorded == [mine]
    assert all(t.recorded == [side] for t in x)


def test_wkv_memory_without_a_given_stream(monkeypatch):
    seen, mine, x, y, s = wkv_forward(monkeypatch, None)
    assert seen["stream"] == 1
    assert len(seen[mine]) == 9 and not y.recorded and not x[0].recorded
