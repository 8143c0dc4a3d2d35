"""GPU tests of state_move: every byte equals the plain gather from the old pool."""
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


def t32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layers,slots,shape,n", [
    (1, 1, (4,), 1), (1, 5, (4,), 5), (3, 7, (4, 5), 7), (2, 40, (2, 64, 64), 40), (1, 300, (3, 60), 300),
    (2, 2000, (4,), 1024), (1, 1024, (36,), 1024), (2, 130, (1, 64, 68), 129), (1, 3, (5, 128, 128), 2),
    (1, 513, (16,), 513), (1, 65, (2048,), 65)])
@pytest.mark.parametrize("kind", ["permute", "fork", "mixed"])
def test_moves(rnn, layers, slots, shape, n, kind):
    r = np.random.default_rng(slots * 7 + n)
    pool = r.normal(size=(layers, slots, *shape)).astype(np.float32)
    dst = r.permutation(slots)[:n]
    if kind == "permute":
        src = r.permutation(dst)
    elif kind == "fork":
        src = np.full(n, r.integers(slots))
    else:  # sources anywhere, freed slots, pairs out of range, targets twice
        src = r.integers(-2, slots + 2, n)
        dst = r.integers(-1, slots + 1, n)
    x = torch.from_numpy(pool).cuda()
    assert rnn.state_move(x, t32(src), t32(dst), slot_dim=1) is x
    np.testing.assert_array_equal(x.cpu().numpy(), gd.move(pool, src, dst))
    if layers == 1:
        y = torch.from_numpy(pool[0]).cuda()
        rnn.state_move(y, t32(src), t32(dst))
        assert torch.equal(y, x[0])


def test_layers_of_a_larger_buffer_and_other_types(rnn):
    base = torch.arange(4 * 3 * 10 * 8, device="cuda", dtype=torch.int32).view(4, 3, 10, 8).to(torch.bfloat16)
    want = base.clone()
    view = base[:, 1]                      # layers apart, slots dense
    rnn.state_move(view, t32([3, -1, 0]), t32([0, 3, 9]), slot_dim=1)
    want[:, 1, 9], want[:, 1, 0], want[:, 1, 3] = want[:, 1, 0].clone(), want[:, 1, 3].clone(), 0
    assert torch.equal(base, want)
    with pytest.raises(ValueError):
        rnn.state_move(base[:, :, 1], t32([0]), t32([1]), slot_dim=1)
    with pytest.raises(rnn.Rwkv7Error):    # 8 bytes per slot
        rnn.state_move(torch.zeros(4, 2, device="cuda"), t32([0]), t32([1]))
    with pytest.raises(rnn.Rwkv7Error):
        rnn.state_move(torch.zeros(4, 4, device="cuda"), t32([0] * 1025), t32([1] * 1025))
    with pytest.raises(ValueError):
        rnn.state_move(torch.zeros(4, 4, device="cuda"), t32([0]), t32([1, 2]))
    x = torch.ones(4, 4, device="cuda")
    rnn.state_move(x, t32([]), t32([]))
    assert x.all()


def test_beams_follow_their_parents_step_after_step(rnn):
    """Ten steps of beam reordering (parents with repeats) in a layer-major pool of WKV7 states."""
    r = np.random.default_rng(4)
    pool = r.normal(size=(3, 16, 2, 64, 64)).astype(np.float32)
    x, dst = torch.from_numpy(pool).cuda(), t32(np.arange(16))
    for _ in range(10):
        src = np.arange(16) // 4 * 4 + r.integers(0, 4, 16)
        rnn.state_move(x, t32(src), dst, slot_dim=1)
        pool = gd.move(pool, src, np.arange(16))
    np.testing.assert_array_equal(x.cpu().numpy(), pool)
