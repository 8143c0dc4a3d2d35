"""Host-side checks of include/gated_delta.h and its binding that need no GPU: every
declared function is exported, sizes are as documented, and bad arguments are refused
before anything is enqueued."""
import ctypes
import os
import re

import pytest

from linear_rnn_sequence_amd import build as hbuild
from linear_rnn_sequence_amd import gated_delta as G
import linear_rnn_sequence_amd as rnn
from tests.test_abi import fake, fake_addresses

pytestmark = pytest.mark.skipif(not os.path.exists(hbuild.LIB),
                                reason="librwkv7_wkv.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")
HEADER = os.path.join(hbuild.INCLUDE, "gated_delta.h")
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE, HIP = range(9)

GATES = ("g", "beta", "dg", "dbeta")  # aligned to their type; everything else to 16 bytes


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b((?:gated_delta|state)_\w+)\s*\(", src))
    assert {"gated_delta_forward", "gated_delta_decode", "gated_delta_forward_train",
            "gated_delta_backward", "state_move"} <= names
    for n in names:
        assert hasattr(ctypes.CDLL(hbuild.LIB), n), n


def test_constants_match_the_header():
    src = open(HEADER).read()
    assert f"#define GATED_DELTA_CHUNK {G.CHUNK}\n" in src
    assert f"#define STATE_MOVE_MAX {G.STATE_MOVE_MAX}\n" in src


def problem(**kw):
    d = dict(n_seq=2, total=16, Hk=2, Hv=4, K=64, V=64, pool=2, scale=0.125, dt=1)
    d.update(kw)
    return G.Problem(**d)


def test_chunks_and_workspaces():
    assert rnn.gated_delta_chunks(0) == 0
    assert rnn.gated_delta_chunks(130, sequences=2) == 4        # two chunks for each 65 tokens
    assert rnn.gated_delta_chunks(130, sequences=2, packed=True) == 130 // 64 + 2
    one = rnn.gated_delta_forward_workspace_bytes(64, 1, 1, 64, 64)
    assert one > 0
    assert rnn.gated_delta_forward_workspace_bytes(640, 2, 4, 64, 128) == 40 * one
    assert rnn.gated_delta_forward_workspace_bytes(0, 2, 4, 64, 128) == 0
    b = rnn.gated_delta_backward_workspace_bytes(64, 1, 1, 128, 64, dtype="f32")
    assert b >= 64 * 128 * 4 + 64 * 64 * 4
    assert rnn.gated_delta_backward_workspace_bytes(64, 1, 1, 96, 64) == 0      # invalid
    with pytest.raises(ValueError):
        rnn.gated_delta_forward_workspace_bytes(64, 1, 1, 64, 64, dtype="fp16")


BAD_PROBLEMS = [
    (dict(dt=2), UNSUPPORTED), (dict(dt=7), DTYPE), (dict(K=96), UNSUPPORTED), (dict(K=256), UNSUPPORTED),
    (dict(V=32), UNSUPPORTED), (dict(V=320), UNSUPPORTED), (dict(V=100), UNSUPPORTED),
    (dict(n_seq=0), SHAPE), (dict(total=-1), SHAPE), (dict(total=15), SHAPE), (dict(Hv=3), SHAPE),
    (dict(Hk=0), SHAPE), (dict(Hv=0), SHAPE), (dict(pool=0), SHAPE), (dict(pool=1), SHAPE),
    (dict(q_stride=127), SHAPE), (dict(k_stride=132), ALIGN), (dict(v_stride=1 << 41), SHAPE),
    (dict(q_stride=-128), SHAPE), (dict(Hk=1 << 26, Hv=1 << 26), SHAPE),
    (dict(n_seq=1 << 20, total=1 << 30, Hk=64, Hv=64, pool=1 << 20), SHAPE),
]


def fwd(p, train=False, over=None, ws=None, ws_bytes=1 << 30, p_ref=True):
    a = dict(q=fake(0), k=fake(1), v=fake(2), g=fake(3), beta=fake(4), s0=fake(5), o=fake(6),
             s_out=fake(7), s_ckpt=fake(8), u=fake(9))
    a.update(over or {})
    ref = ctypes.byref(p) if p_ref else None
    ws = fake(12) if ws is None else (None if ws == 0 else ws)
    names = ["q", "k", "v", "g", "beta", "s0", "o", "s_out"] + (["s_ckpt", "u"] if train else [])
    fn = G.lib().gated_delta_forward_train if train else G.lib().gated_delta_forward
    return fn(ref, *(a[n] for n in names), ws, ws_bytes, None)


@fake_addresses
@pytest.mark.parametrize("change,code", BAD_PROBLEMS)
def test_bad_problems(change, code):
    assert fwd(problem(**change)) == code
    assert fwd(problem(**change), train=True) == code
    assert bwd(problem(**change)) == code
    assert G.lib().gated_delta_forward_workspace(ctypes.byref(problem(**change))) == 0


@fake_addresses
@pytest.mark.parametrize("train", [False, True])
def test_forward_refusals(train):
    p = problem()
    assert fwd(p, train, p_ref=False) == NULL
    for n in ("q", "k", "v", "g", "beta", "o") + (("s_ckpt", "u") if train else ()):
        assert fwd(p, train, {n: None}) == NULL, n
        assert fwd(p, train, {n: fake(20, 1 if n in GATES else 8)}) == ALIGN, n
    assert fwd(p, train, {"s0": fake(5, 4)}) == ALIGN
    assert fwd(p, train, {"s_out": fake(5, 64)}) == ALIAS      # part of s0
    for n in ("q", "k", "v", "g", "beta", "s0", "s_out"):
        i = dict(q=0, k=1, v=2, g=3, beta=4, s0=5, s_out=7)[n]
        assert fwd(p, train, {"o": fake(i, 16)}) == ALIAS, n
    assert fwd(p, train, ws=0) == WORKSPACE
    assert fwd(p, train, ws_bytes=100) == WORKSPACE
    assert fwd(p, train, ws=fake(12, 8)) == ALIGN
    assert fwd(p, train, ws=fake(6)) == ALIAS
    if train:
        assert fwd(p, train, {"u": fake(6)}) == ALIAS
        assert fwd(problem(slots_in=fake(15).value), train) == UNSUPPORTED


@fake_addresses
def test_index_arrays_are_aligned_and_not_written():
    assert fwd(problem(cu_seqlens=fake(15, 2).value)) == ALIGN
    assert fwd(problem(slots_in=fake(15, 1).value, slots_out=fake(15).value)) == ALIGN
    assert fwd(problem(cu_seqlens=fake(6).value)) == ALIAS
    assert fwd(problem(slots_in=fake(14).value, slots_out=fake(7).value)) == ALIAS


def bwd(p, over=None, ws=None, ws_bytes=1 << 40):
    names = ["q", "k", "v", "g", "beta", "d_o", "s_ckpt", "u", "ds_T", "dq", "dk", "dv", "dg", "dbeta", "ds0"]
    a = {n: fake(i) for i, n in enumerate(names)}
    a.update(over or {})
    ws = fake(20) if ws is None else (None if ws == 0 else ws)
    return G.lib().gated_delta_backward(ctypes.byref(p), *(a[n] for n in names), ws, ws_bytes, None)


@fake_addresses
def test_backward_refusals():
    p = problem()
    names = ["q", "k", "v", "g", "beta", "d_o", "s_ckpt", "u", "ds_T", "dq", "dk", "dv", "dg", "dbeta", "ds0"]
    for n in names:
        if n not in ("ds_T", "ds0"):
            assert bwd(p, {n: None}) == NULL, n
        assert bwd(p, {n: fake(25, 1 if n in GATES else 8)}) == ALIGN, n
    for i, n in enumerate(names[:9]):
        assert bwd(p, {"dq": fake(i)}) == ALIAS, n
    assert bwd(p, {"dk": fake(9, 16)}) == ALIAS
    assert bwd(p, {"ds0": fake(8, 16)}) == ALIAS               # part of ds_T
    assert bwd(p, ws=0) == WORKSPACE and bwd(p, ws_bytes=1) == WORKSPACE
    assert bwd(p, ws=fake(13)) == ALIAS
    assert bwd(problem(slots_out=fake(30).value)) == UNSUPPORTED


@fake_addresses
def test_decode_refusals():
    def dec(p, **over):
        a = dict(q=fake(0), k=fake(1), v=fake(2), g=fake(3), beta=fake(4), state=fake(5), o=fake(6))
        a.update(over)
        return G.lib().gated_delta_decode(ctypes.byref(p), *a.values(), None)

    p = problem(total=2)
    for n in ("q", "k", "v", "g", "beta", "state", "o"):
        assert dec(p, **{n: None}) == NULL, n
        assert dec(p, **{n: fake(9, 1 if n in GATES else 4)}) == ALIGN, n
    assert dec(problem(total=4)) == SHAPE                       # two tokens each
    assert dec(problem(total=2, cu_seqlens=fake(11).value)) == SHAPE
    assert dec(problem(total=2, slots_in=fake(11).value)) == SHAPE
    assert dec(p, o=fake(5, 64)) == ALIAS and dec(p, state=fake(1)) == ALIAS
    assert dec(problem(total=2, K=32)) == UNSUPPORTED


@fake_addresses
def test_move_refusals():
    def mv(pool=fake(0), layers=2, layer=1 << 20, slots=4, size=256, src=fake(1), dst=fake(2), n=3):
        return G.lib().state_move(pool, layers, layer, slots, size, src, dst, n, None)

    assert mv(pool=None) == NULL and mv(src=None) == NULL and mv(dst=None) == NULL
    assert mv(n=0, pool=None) == OK
    for bad in (dict(layers=0), dict(slots=0), dict(n=-1), dict(n=1025), dict(size=0), dict(size=24),
                dict(layer=512), dict(layer=(1 << 20) + 8), dict(size=1 << 62), dict(layer=1 << 62, layers=8)):
        assert mv(**bad) == SHAPE, bad
    assert mv(pool=fake(0, 8)) == ALIGN and mv(src=fake(1, 2)) == ALIGN
    assert mv(dst=fake(0, (1 << 20) + 16)) == ALIAS             # inside the second layer


def test_binding_refuses_what_is_not_on_a_gpu_or_has_wrong_shapes():
    x = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q, v, g = x(1, 4, 2, 64), x(1, 4, 4, 64), x(1, 4, 4)
    with pytest.raises(ValueError, match="GPU"):
        rnn.gated_delta_forward(q, q, v, g, g)
    with pytest.raises(TypeError):
        rnn.gated_delta_forward(q.half(), q.half(), v.half(), g.half(), g.half())
    with pytest.raises(ValueError):
        rnn.gated_delta_forward(q[0], q[0], v[0], g[0], g[0])
    with pytest.raises(ValueError):
        rnn.gated_delta_forward(q, q, v, g, g, slots_in=g)
    with pytest.raises(ValueError):
        rnn.gated_delta_decode(q, q, v, g, g, torch.zeros(1, 4, 64, 64))
    with pytest.raises(ValueError, match="GPU"):
        rnn.state_move(torch.zeros(4, 64), g, g)
    with pytest.raises(ValueError):
        rnn.state_move(torch.zeros(4), g, g, slot_dim=2)


def test_token_strides():
    base = torch.zeros(2, 5, 7, 64, dtype=torch.bfloat16)
    assert G._token_stride(base, "q", (2, 5), 7, 64) == 0
    assert G._token_stride(base[:, :, 2:5], "q", (2, 5), 3, 64) == 7 * 64
    assert G._token_stride(base[:1, :, :1], "q", (1, 5), 1, 64) == 7 * 64
    assert G._token_stride(base[:, :1, 2:5], "q", (2, 1), 3, 64) == 5 * 7 * 64
    assert G._token_stride(base[:, 2], "q", (2,), 7, 64) == 5 * 7 * 64
    for bad in (base[:, :3], base.transpose(1, 2), base[..., ::2]):
        with pytest.raises(ValueError):
            G._token_stride(bad, "q", tuple(bad.shape[:2]), *bad.shape[2:])


def test_tokens_in_each_others_place_are_refused():
    """One token shown as several (a stride of nothing, which the library takes for dense rows), and
    windows that overlap."""
    one = torch.zeros(1, 1, 7, 64, dtype=torch.bfloat16)
    flat = torch.zeros(4096, dtype=torch.bfloat16)
    for bad in (one.expand(1, 5, 7, 64), one.expand(2, 5, 7, 64), flat.as_strided((1, 5, 7, 64), (4096, 64, 64, 1))):
        with pytest.raises(ValueError):
            G._token_stride(bad, "q", tuple(bad.shape[:2]), *bad.shape[2:])
    for bad in (one[0].expand(5, 7, 64), flat.as_strided((5, 7, 64), (64, 64, 1))):
        with pytest.raises(ValueError):
            G._token_stride(bad, "q", (5,), 7, 64)
    assert G._token_stride(one[..., :3, :], "q", (1, 1), 3, 64) in (0, 3 * 64)
    assert G._token_stride(one[:0], "q", (0, 1), 7, 64) in (0, 7 * 64)


def test_stored_states_need_the_bits_behind_them():
    """bf16 states lie 5/4 V K apart; a copy without what lies behind them, and a view whose memory ends with the
    last state, are refused on the host."""
    cpu, tail, chunks = torch.device("cpu"), (2, 64, 128), 3
    size = G._ckpt_size(torch, 64, 128, torch.bfloat16)
    assert size == 64 * 128 * 5 // 4 and G._ckpt_size(torch, 64, 128, torch.float32) == 64 * 128
    strides = (2 * size, size, 128, 1)
    whole = torch.zeros(chunks * 2 * size, dtype=torch.bfloat16)
    good = whole.as_strided((chunks, *tail), strides)
    G._check_ckpt(torch, good, chunks, tail, torch.bfloat16, cpu)
    short = torch.zeros(chunks * 2 * size - 64 * 32, dtype=torch.bfloat16).as_strided((chunks, *tail), strides)
    for bad in (good.contiguous(), good[1:], short, good.float()):
        with pytest.raises(ValueError):
            G._check_ckpt(torch, bad, chunks, tail, torch.bfloat16, cpu)
    with pytest.raises(ValueError):  # the same rows, further on in the memory
        G._check_ckpt(torch, whole.as_strided((2, *tail), strides, 2 * size + 128), 2, tail, torch.bfloat16, cpu)
    G._check_ckpt(torch, torch.zeros(chunks, *tail), chunks, tail, torch.float32, cpu)


def test_moves_read_each_pair_once():
    """The kernel searches a table for the targets it has put there; a second read of the list, written meanwhile,
    could give one that is not, and the search would not end."""
    src = re.sub(r"//.*", "", open(os.path.join(hbuild.CSRC, "state_move.hip")).read())
    for name in ("src", "dst"):
        assert len(re.findall(rf"\bp\.{name}\[", src)) == 1, name


@pytest.mark.parametrize("dtype,name", [(torch.bfloat16, "bf16"), (torch.float32, "f32")])
def test_stored_states_as_one_dense_tensor(dtype, name):
    """[chunks, Hv, GATED_DELTA_CKPT_SIZE], which may be copied; other sizes, types and layouts are refused."""
    cpu, tail, chunks = torch.device("cpu"), (2, 64, 128), 3
    size = rnn.gated_delta_ckpt_size(64, 128, dtype=name)
    assert size == G._ckpt_size(torch, 64, 128, dtype)
    good = torch.zeros(chunks, 2, size, dtype=dtype)
    G._check_ckpt(torch, good, chunks, tail, dtype, cpu)
    G._check_ckpt(torch, good.clone(), chunks, tail, dtype, cpu)
    for bad in (good[1:], good[:, :1], good[..., :-1], good.transpose(0, 1), torch.zeros(chunks, 2, size + 4, dtype=dtype)):
        with pytest.raises(ValueError):
            G._check_ckpt(torch, bad, chunks, tail, dtype, cpu)
    with pytest.raises(TypeError):
        G._check_ckpt(torch, good.half(), chunks, tail, dtype, cpu)


class Wide:
    """A tensor of any size, without its memory."""

    def __init__(self, shape, dtype=torch.float32):
        self.shape, self.dtype, self.device = shape, dtype, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return 4 if self.dtype == torch.float32 else 2

    def data_ptr(self):
        raise AssertionError("refused before")


def test_numbers_that_do_not_fit_an_int_are_refused():
    """2^32 + 4 slots of 16 bytes would be 4 to the library, 2^32 + 1 sequences one."""
    pair = Wide((2,), torch.int32)
    for shape, dim in (((2 ** 32 + 4, 4), 0), ((1, 2 ** 32 + 4, 4), 1), ((2 ** 32 + 1, 2, 4), 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            rnn.state_move(Wide(shape), pair, pair, slot_dim=dim)
    with pytest.raises(ValueError, match="2\\^31"):
        rnn.state_move(Wide((4, 4)), Wide((2 ** 32 + 1,), torch.int32), Wide((2 ** 32 + 1,), torch.int32))
    bf = torch.bfloat16
    for T, n in ((2 ** 32 + 64, 2), (64, 2 ** 32 + 1)):
        q, v, g = Wide((1, T, 1, 64), bf), Wide((1, T, 1, 64), bf), Wide((1, T, 1), bf)
        with pytest.raises(ValueError, match="2\\^31"):
            rnn.gated_delta_forward(q, q, v, g, g, cu_seqlens=Wide((n + 1,), torch.int32), want_state=False)
    for f in (rnn.gated_delta_forward_workspace_bytes, rnn.gated_delta_backward_workspace_bytes):
        with pytest.raises(ValueError, match="2\\^31"):
            f(2 ** 32 + 64, 1, 1, 64, 64)
    with pytest.raises(ValueError, match="2\\^31"):
        rnn.gated_delta_chunks(2 ** 33)
    assert rnn.gated_delta_forward_workspace_bytes(-1, 1, 1, 64, 64) == 0  # invalid, as other sizes that are none
