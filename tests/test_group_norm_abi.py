"""The float64 group norm against torch and differences, and host-side checks of include/group_norm.h
and its binding that need no GPU."""
import ctypes
import os
import re

import numpy as np
import pytest

from linear_rnn_sequence_amd import build as hbuild
from linear_rnn_sequence_amd import group_norm as N
import linear_rnn_sequence_amd as rnn
from oracle import group_norm as gn
from tests.test_abi import fake, fake_addresses
from tests.test_gated_delta_abi import Wide

pytestmark = pytest.mark.skipif(not os.path.exists(hbuild.LIB),
                                reason="librwkv7_wkv.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")
HEADER = os.path.join(hbuild.INCLUDE, "group_norm.h")
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE, HIP = range(9)


# ------------------------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", list(N.ACTIVATIONS))
def test_forward_against_torch(act, gated):
    r = np.random.default_rng(1)
    x, z, w, b = r.normal(size=(5, 12)), r.normal(size=(5, 12)), r.normal(size=12), r.normal(size=12)
    f = {"none": lambda t: t, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[act]
    t = [torch.from_numpy(a) for a in (x, w, b, z)]
    n = torch.nn.functional.group_norm(t[0], 3, t[1], t[2], 1e-5)
    want = n * f(t[3]) if gated else f(n)
    got = gn.forward(x, 3, weight=w, bias=b, gate=z if gated else None, activation=act)
    np.testing.assert_allclose(got, want.numpy(), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", list(N.ACTIVATIONS))
def test_gradients_against_differences(act, gated, rms):
    r = np.random.default_rng(2)
    p = dict(x=r.normal(size=(2, 6)), weight=r.normal(size=6), bias=r.normal(size=6), gate=r.normal(size=(2, 6)))
    if not gated:
        del p["gate"]
    dy = r.normal(size=(2, 6))

    def loss(q):
        q = dict(q)
        return (gn.forward(q.pop("x"), 2, activation=act, rms=rms, **q) * dy).sum()

    rest = {n: a for n, a in p.items() if n != "x"}
    grads = gn.backward(p["x"], 2, dy, activation=act, rms=rms, **rest)
    for n, d in zip(("x", "weight", "bias", "gate"), grads):
        if d is None:
            continue
        for at in np.ndindex(*d.shape):
            lo, hi = ({**p, n: p[n].copy()} for _ in range(2))
            lo[n][at] -= 1e-5
            hi[n][at] += 1e-5
            # central differences: (1e-5)^2 of the third derivative, and 1e-16 / 1e-5 of the loss
            assert abs((loss(hi) - loss(lo)) / 2e-5 - d[at]) < 1e-7 * max(1, np.abs(d).max()), (n, at)


# ------------------------------------------------------------------------------------ the library

def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(group_norm_\w+)\s*\(", src))
    assert names == {"group_norm_forward", "group_norm_backward", "group_norm_backward_workspace"}
    for n in names:
        assert hasattr(ctypes.CDLL(hbuild.LIB), n), n


def test_the_header_and_the_binding_agree():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{(.*?)\} group_norm_problem;", src, re.S).group(1)
    assert re.findall(r"(\w+)\s*[,;]", body) == [n for n, _ in N.Problem._fields_]
    for name, code in N.ACTIVATIONS.items():
        assert f"GROUP_NORM_{name.upper()} = {code}" in src
    assert f"kMaxSize = {N.MAX_SIZE};" in open(os.path.join(hbuild.CSRC, "group_norm.hip")).read()


def problem(**kw):
    d = dict(rows=10, groups=4, size=64, eps=1e-5, activation=1, dt=1)
    d.update(kw)
    return N.Problem(**d)


BAD_PROBLEMS = [
    (dict(dt=2), UNSUPPORTED), (dict(dt=7), DTYPE), (dict(activation=3), UNSUPPORTED), (dict(activation=-1), UNSUPPORTED),
    (dict(size=1025), UNSUPPORTED), (dict(size=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=-4), SHAPE),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(groups=1 << 17, size=128), SHAPE),
    (dict(x_stride=255), SHAPE), (dict(gate_stride=255), SHAPE), (dict(x_stride=-256), SHAPE),
    (dict(x_stride=(1 << 23) + 8), SHAPE), (dict(gate_stride=1 << 41), SHAPE), (dict(groups=1 << 30, size=1024), SHAPE),
]

FWD = ["x", "gate", "weight", "bias", "y"]
BWD = ["x", "gate", "weight", "bias", "dy", "dx", "dgate", "dweight", "dbias"]


def fwd(p, over=None, ref=True):
    a = {n: fake(i) for i, n in enumerate(FWD)} | (over or {})
    return N.lib().group_norm_forward(ctypes.byref(p) if ref else None, *a.values(), None)


def bwd(p, over=None, ws=None, ws_bytes=1 << 30):
    a = {n: fake(i) for i, n in enumerate(BWD)} | (over or {})
    ws = fake(12) if ws is None else (None if ws == 0 else ws)
    return N.lib().group_norm_backward(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


@fake_addresses
@pytest.mark.parametrize("change,code", BAD_PROBLEMS)
def test_bad_problems(change, code):
    assert fwd(problem(**change)) == code
    assert bwd(problem(**change)) == code
    assert N.lib().group_norm_backward_workspace(ctypes.byref(problem(**change))) == 0


@fake_addresses
def test_forward_refusals():
    p = problem()
    assert fwd(p, ref=False) == NULL
    for n in FWD:
        if n in ("x", "y"):
            assert fwd(p, {n: None}) == NULL, n
        assert fwd(p, {n: fake(9, 2 if n in ("weight", "bias") else 1)}) == ALIGN, n
    for i, n in enumerate(FWD[1:4], 1):
        assert fwd(p, {"y": fake(i)}) == ALIAS, n
    assert fwd(p, {"y": fake(0, 16)}) == ALIAS
    assert fwd(problem(x_stride=300), {"y": fake(0)}) == ALIAS      # in place, but strided
    assert fwd(problem(rows=0), {"x": None, "y": None}) == OK


@fake_addresses
def test_backward_refusals():
    p = problem()
    for n in ("x", "dy", "dx", "gate", "dgate"):
        assert bwd(p, {n: None}) == NULL, n
    for n in BWD:
        small = n in ("weight", "bias", "dweight", "dbias")
        assert bwd(p, {n: fake(20, 2 if small else 1)}) == ALIGN, n
    for i, n in enumerate(BWD[:4]):
        assert bwd(p, {"dx": fake(i)}) == ALIAS, n
        assert bwd(p, {"dweight": fake(i)}) == ALIAS, n
    assert bwd(p, {"dx": fake(4, 16)}) == ALIAS and bwd(p, {"dgate": fake(4)}) == ALIAS
    assert bwd(p, {"dgate": fake(5)}) == ALIAS and bwd(p, {"dbias": fake(7, 16)}) == ALIAS
    assert bwd(p, ws=0) == WORKSPACE and bwd(p, ws_bytes=100) == WORKSPACE
    assert bwd(p, ws=fake(12, 8)) == ALIGN and bwd(p, ws=fake(5)) == ALIAS


def test_workspace():
    # two rows of [C] for every workgroup's rows: four each for its eight teams to a group
    assert rnn.group_norm_backward_workspace_bytes(8, 4, 64) == 2 * 256 * 4
    assert rnn.group_norm_backward_workspace_bytes(32, 4, 64) == 2 * 256 * 4
    assert rnn.group_norm_backward_workspace_bytes(33, 4, 64) == 2 * 2 * 256 * 4
    assert rnn.group_norm_backward_workspace_bytes(0, 4, 64) == 0
    assert rnn.group_norm_backward_workspace_bytes(1 << 20, 32, 128) <= (1 << 20) * 32 * 128 * 2 // 4
    assert rnn.group_norm_backward_workspace_bytes(8, 4, 2000) == 0  # invalid
    with pytest.raises(ValueError):
        rnn.group_norm_backward_workspace_bytes(8, 1 << 40, 1)


def test_binding_refuses():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        rnn.group_norm_forward(x, 2)
    with pytest.raises(TypeError):
        rnn.group_norm_forward(x.half(), 2)
    g = Wide((2, 3, 64), torch.bfloat16)
    for kw, error in ((dict(groups=3), "equal groups"), (dict(groups=0), "equal groups"),
                      (dict(groups=-2), "equal groups"), (dict(groups=2, activation="gelu"), "activation"),
                      (dict(groups=2, weight=Wide((63,))), "weight"), (dict(groups=2, gate=Wide((2, 64), torch.bfloat16)), "gate"),
                      (dict(groups=2, y=Wide((2, 3, 32), torch.bfloat16)), "y")):
        with pytest.raises(ValueError, match=error):
            rnn.group_norm_forward(g, **kw)
    for kw in (dict(weight=Wide((64,), torch.bfloat16)), dict(gate=Wide((2, 3, 64)))):
        with pytest.raises(TypeError):
            rnn.group_norm_forward(g, 2, **kw)
    with pytest.raises(ValueError, match="at most"):
        rnn.group_norm_forward(Wide((2, 2048), torch.bfloat16), 1)
    for kw, error in ((dict(dy=None), "dy"), (dict(dgate=g), "dgate"), (dict(dweight=Wide((64,))), "dweight"),
                      (dict(dbias=Wide((64,))), "dbias")):
        with pytest.raises(ValueError, match=error):
            rnn.group_norm_backward(g, 2, **({"dy": g} | kw))


def test_row_strides():
    base = torch.zeros(2, 5, 100)
    assert N._row_stride(base, "x", base.shape) == 0
    part = base[..., 10:74]
    assert N._row_stride(part, "x", part.shape) == 100
    assert N._row_stride(part[0], "x", (5, 64)) == 100
    assert N._row_stride(part[:, 1], "x", (2, 64)) == 500
    assert N._row_stride(part[:1, :1], "x", (1, 1, 64)) in (0, 64, 100)
    assert N._row_stride(part[:, :1], "x", (2, 1, 64)) == 500
    flat = torch.zeros(640)
    for bad in (base[:, :3, 10:74], base.transpose(0, 1), base[..., ::2], base[:1, :1].expand(2, 5, 100),
                flat.as_strided((5, 64), (32, 1)), base[0, 0, :64].expand(5, 64)):
        with pytest.raises(ValueError):
            N._row_stride(bad, "x", bad.shape)
