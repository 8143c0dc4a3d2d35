"""Host-side checks of include/linear_attention.h and its binding that need no GPU: every declared
function is exported, sizes are as documented, and bad arguments are refused before anything is
enqueued."""
import ctypes
import os
import re

import pytest

from linear_rnn_sequence_amd import build as hbuild
from linear_rnn_sequence_amd import linear_attention as A
import linear_rnn_sequence_amd as rnn
from tests.test_abi import fake, fake_addresses
from tests.test_gated_delta_abi import Wide

pytestmark = pytest.mark.skipif(not os.path.exists(hbuild.LIB),
                                reason="librwkv7_wkv.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")
HEADER = os.path.join(hbuild.INCLUDE, "linear_attention.h")
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE, HIP = range(9)

FLOATS = ("g", "dg")  # aligned to their type; everything else to 16 bytes


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(linear_attention_\w+)\s*\(", src))
    assert len(names) == 5
    for n in names:
        assert hasattr(ctypes.CDLL(hbuild.LIB), n), n


def test_the_problem_has_the_headers_fields():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{(.*?)\} linear_attention_problem;", src, re.S).group(1)
    names = re.findall(r"(\w+)\s*[,;]", body)
    assert names == [n for n, _ in A.Problem._fields_]


def problem(**kw):
    d = dict(n_seq=2, total=16, Hk=2, Hv=4, K=64, V=64, pool=2, scale=0.125, dt=1)
    d.update(kw)
    return A.Problem(**d)


def test_workspaces():
    assert rnn.linear_attention_forward_workspace_bytes(64, 1, 1, 64, 64) == 0     # one segment
    assert rnn.linear_attention_forward_workspace_bytes(0, 2, 4, 64, 128) == 0
    # a long sequence in segments: a state each
    assert rnn.linear_attention_forward_workspace_bytes(1 << 15, 1, 1, 64, 128) % (64 * 128 * 4) == 0
    assert rnn.linear_attention_forward_workspace_bytes(1 << 15, 1, 1, 64, 128) > 0
    for tokens in range(200, 800, 7):  # around the shortest segment
        for packed in (False, True):
            got = rnn.linear_attention_forward_workspace_bytes(2 * tokens, 1, 2, 64, 64, sequences=2, packed=packed)
            assert got % (2 * 64 * 64 * 4) == 0
    # the backward: a number for dg for every head (of at most 128 values), shared heads' gradients
    assert rnn.linear_attention_backward_workspace_bytes(64, 2, 2, 64, 64) == 2 * 8
    assert rnn.linear_attention_backward_workspace_bytes(64, 1, 1, 64, 192) == 2 * 64 * 3 * 64 * 4 + 3 * 8
    assert rnn.linear_attention_backward_workspace_bytes(64, 1, 2, 128, 256, sequences=4) == \
        2 * 64 * 4 * 128 * 4 + 4 * 4 * 8
    assert rnn.linear_attention_backward_workspace_bytes(64, 1, 1, 96, 64) == 0      # invalid
    with pytest.raises(ValueError):
        rnn.linear_attention_forward_workspace_bytes(64, 1, 1, 64, 64, dtype="fp16")


BAD_PROBLEMS = [
    (dict(dt=2), UNSUPPORTED), (dict(dt=7), DTYPE), (dict(K=96), UNSUPPORTED), (dict(K=256), UNSUPPORTED),
    (dict(V=32), UNSUPPORTED), (dict(V=320), UNSUPPORTED), (dict(V=100), UNSUPPORTED),
    (dict(n_seq=0), SHAPE), (dict(total=-1), SHAPE), (dict(total=15), SHAPE), (dict(Hv=3), SHAPE),
    (dict(Hk=0), SHAPE), (dict(Hv=0), SHAPE), (dict(pool=0), SHAPE), (dict(pool=1), SHAPE),
    (dict(q_stride=127), SHAPE), (dict(k_stride=132), ALIGN), (dict(v_stride=1 << 41), SHAPE),
    (dict(q_stride=-128), SHAPE), (dict(Hk=1 << 26, Hv=1 << 26), SHAPE),
    (dict(Hk=1, Hv=1 << 16, K=128, V=192), SHAPE),      # rows of a key head's gradients above 2^23
    (dict(n_seq=1 << 20, total=1 << 30, Hk=64, Hv=64, pool=1 << 20), SHAPE),
    (dict(n_seq=1 << 20, total=1 << 30, Hk=64, Hv=64, pool=1 << 20, cu_seqlens=1 << 12), SHAPE),
]


def fwd(p, over=None, ws=None, ws_bytes=1 << 30, p_ref=True):
    a = dict(q=fake(0), k=fake(1), v=fake(2), g=fake(3), s0=fake(5), o=fake(6), s_out=fake(7))
    a.update(over or {})
    ws = fake(12) if ws is None else (None if ws == 0 else ws)
    return A.lib().linear_attention_forward(ctypes.byref(p) if p_ref else None, *a.values(), ws, ws_bytes, None)


BWD = ["q", "k", "v", "g", "d_o", "s0", "ds_T", "dq", "dk", "dv", "dg", "ds0"]


def bwd(p, over=None, ws=None, ws_bytes=1 << 40):
    a = {n: fake(i) for i, n in enumerate(BWD)}
    a.update(over or {})
    ws = fake(20) if ws is None else (None if ws == 0 else ws)
    return A.lib().linear_attention_backward(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


@fake_addresses
@pytest.mark.parametrize("change,code", BAD_PROBLEMS)
def test_bad_problems(change, code):
    assert fwd(problem(**change)) == code
    assert bwd(problem(**change)) == code
    assert A.lib().linear_attention_forward_workspace(ctypes.byref(problem(**change))) == 0
    assert A.lib().linear_attention_backward_workspace(ctypes.byref(problem(**change))) == 0


@fake_addresses
def test_forward_refusals():
    p = problem()
    assert fwd(p, p_ref=False) == NULL
    for n in ("q", "k", "v", "g", "o"):
        assert fwd(p, {n: None}) == NULL, n
        assert fwd(p, {n: fake(20, 1 if n in FLOATS else 8)}) == ALIGN, n
    assert fwd(problem(total=0), {"g": None}) == NULL
    assert fwd(p, {"s0": fake(5, 4)}) == ALIGN
    assert fwd(p, {"s_out": fake(5, 64)}) == ALIAS      # part of s0
    for n, i in dict(q=0, k=1, v=2, g=3, s0=5, s_out=7).items():
        assert fwd(p, {"o": fake(i)}) == ALIAS, n
    assert fwd(p, {"s0": fake(7), "o": fake(7, 256)}) == ALIAS
    long = problem(n_seq=1, total=1 << 15, pool=1)
    need = A.lib().linear_attention_forward_workspace(ctypes.byref(long))
    assert need > 0 and fwd(long, ws=0) == WORKSPACE and fwd(long, ws_bytes=need - 1) == WORKSPACE
    assert fwd(long, ws=fake(12, 8)) == ALIGN
    assert fwd(long, ws=fake(6)) == ALIAS
    assert fwd(long, {"s0": fake(7)}, ws=fake(7)) == ALIAS


@fake_addresses
def test_index_arrays_are_aligned_and_not_written():
    assert fwd(problem(cu_seqlens=fake(15, 2).value)) == ALIGN
    assert fwd(problem(slots_in=fake(15, 1).value, slots_out=fake(15).value)) == ALIGN
    assert fwd(problem(cu_seqlens=fake(6).value)) == ALIAS
    assert fwd(problem(slots_in=fake(14).value, slots_out=fake(7).value)) == ALIAS


@fake_addresses
def test_backward_refusals():
    p = problem()
    for n in BWD:
        if n not in ("s0", "ds_T", "dg", "ds0"):
            assert bwd(p, {n: None}) == NULL, n
        assert bwd(p, {n: fake(25, 1 if n in FLOATS else 8)}) == ALIGN, n
    for i, n in enumerate(BWD[:7]):
        assert bwd(p, {"dq": fake(i)}) == ALIAS, n
    assert bwd(p, {"dk": fake(7, 16)}) == ALIAS
    assert bwd(p, {"dg": fake(3)}) == ALIAS
    assert bwd(p, {"ds0": fake(6, 16)}) == ALIAS               # part of ds_T
    assert bwd(p, {"ds0": fake(5)}) == ALIAS                   # s0
    assert bwd(p, ws=0) == WORKSPACE and bwd(p, ws_bytes=1) == WORKSPACE
    assert bwd(p, ws=fake(9)) == ALIAS
    assert bwd(problem(slots_out=fake(30).value)) == UNSUPPORTED


@fake_addresses
def test_decode_refusals():
    def dec(p, **over):
        a = dict(q=fake(0), k=fake(1), v=fake(2), g=fake(3), state=fake(5), o=fake(6))
        a.update(over)
        return A.lib().linear_attention_decode(ctypes.byref(p), *a.values(), None)

    p = problem(total=2)
    for n in ("q", "k", "v", "g", "state", "o"):
        assert dec(p, **{n: None}) == NULL, n
        assert dec(p, **{n: fake(9, 1 if n in FLOATS else 4)}) == ALIGN, n
    assert dec(problem(total=4)) == SHAPE                       # two tokens each
    assert dec(problem(total=2, cu_seqlens=fake(11).value)) == SHAPE
    assert dec(problem(total=2, slots_in=fake(11).value)) == SHAPE
    assert dec(p, o=fake(5, 64)) == ALIAS and dec(p, state=fake(1)) == ALIAS
    assert dec(problem(total=2, K=32)) == UNSUPPORTED


def test_binding_refuses_what_is_not_on_a_gpu_or_has_wrong_shapes():
    x = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q, v, g = x(1, 4, 2, 64), x(1, 4, 4, 64), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        rnn.linear_attention_forward(q, q, v, g)
    with pytest.raises(TypeError):
        rnn.linear_attention_forward(q.half(), q.half(), v.half(), g)
    with pytest.raises(ValueError):
        rnn.linear_attention_forward(q[0], q[0], v[0], g)
    with pytest.raises(ValueError):
        rnn.linear_attention_forward(q, q, v, g, slots_in=g)
    with pytest.raises(ValueError):
        rnn.linear_attention_decode(q, q, v, g, torch.zeros(1, 4, 64, 64))
    with pytest.raises(ValueError, match="state"):
        rnn.linear_attention_decode(q[0], q[0], v[0], g, None)


def on_gpu(*shape, dtype=torch.bfloat16):
    return Wide(shape, dtype)


def test_binding_refuses_wrong_gates_and_types():
    q, v = on_gpu(1, 4, 2, 64), on_gpu(1, 4, 4, 64)
    for g in (on_gpu(2, dtype=torch.float32), on_gpu(1, 4, 4, dtype=torch.float32)):
        with pytest.raises(ValueError, match="^g"):
            rnn.linear_attention_forward(q, q, v, g)
    with pytest.raises(TypeError, match="^g"):
        rnn.linear_attention_forward(q, q, v, on_gpu(4))
    g = on_gpu(4, dtype=torch.float32)
    with pytest.raises(TypeError):
        rnn.linear_attention_forward(q, q, on_gpu(1, 4, 4, 64, dtype=torch.float32), g)
    with pytest.raises(ValueError, match="^k"):
        rnn.linear_attention_forward(q, on_gpu(1, 5, 2, 64), v, g)
    with pytest.raises(ValueError, match="B = 1"):
        rnn.linear_attention_forward(on_gpu(2, 4, 2, 64), on_gpu(2, 4, 2, 64), on_gpu(2, 4, 4, 64), g,
                                     cu_seqlens=on_gpu(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="d_o"):
        rnn.linear_attention_backward(q, q, v, g, None)
    with pytest.raises(ValueError, match="2\\^31"):
        rnn.linear_attention_forward(on_gpu(1, 2 ** 32 + 64, 1, 64), on_gpu(1, 2 ** 32 + 64, 1, 64),
                                     on_gpu(1, 2 ** 32 + 64, 4, 64), g)
    for f in (rnn.linear_attention_forward_workspace_bytes, rnn.linear_attention_backward_workspace_bytes):
        with pytest.raises(ValueError, match="2\\^31"):
            f(2 ** 32 + 64, 1, 1, 64, 64)
        assert f(-1, 1, 1, 64, 64) == 0


@pytest.mark.parametrize("heads,K,V", [(64, 64, 64), (64, 128, 256), (64, 64, 192), (32, 128, 128)])
def test_large_batches_are_taken(heads, K, V):
    """All whose states are below 2^38 bytes, whole or in segments."""
    sequences = 2 ** 38 // (4 * heads * K * V)
    sequences -= 2 ** 38 % (4 * heads * K * V) == 0
    size = lambda n, packed: rnn.linear_attention_backward_workspace_bytes(  # noqa: E731
        n, heads, heads, K, V, sequences=n, packed=packed)
    parts = {64: 1, 128: 1, 192: 3, 256: 2}[V]
    for n in (2048, 4096, 8192, sequences):
        for packed in (False, True):  # (a number for dg for each, and where V is in parts gradients to add)
            assert size(n, packed) == n * heads * parts * 8 + (2 * n * heads * parts * K * 4 if parts > 1 else 0)
    assert size(sequences + 1, False) == 0
