"""GPU parity of the group norm with its float64 implementation, at the sizes, strides and values where
it can go wrong; and of the layer that it ends: linear attention, norm and gate, forward and backward.

Tolerances (2-norm of the difference over that of the result, and the largest over the largest):
 - float32: about ten roundings of 2^-24 per value and sums of up to 1024 terms, the exponential's
   2^-22: 1e-6 and 4e-6.
 - bf16: rounded once, 2^-8 = 3.9e-3; what it is rounded from is 2^-20 off.
 - dweight, dbias: float32 sums over the rows of terms of either sign, compared with the sums of their
   sizes: sqrt(rows) 2^-24 for the roundings of the sum and 2^-21 for the terms' own errors, about eight
   roundings.  The size of a term is that of what it is formed from: u is a difference, off by 2^-24 of
   (|x| + |mean|) rstd however small it is itself, and without a gate silu' = s + n (s - s^2) one too, of
   parts below 1 + |n|.
"""
import numpy as np
import pytest

from oracle import group_norm as gn
from oracle import linear_attention as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NORM = {"f32": 1e-6, "bf16": 4e-3}
LARGEST = {"f32": 4e-6, "bf16": 4e-3}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def rnn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_rnn_sequence_amd as m

    m.lib()
    return m


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(13)


def f64(x):
    return None if x is None else x.detach().to("cpu", torch.float64).numpy()


def close(got, want, dtype, what, terms=None):
    """``terms``: the sizes of what an output is the difference of (a group of two channels has u = +1 and -1
    but for eps, and the terms of dx cancel): eight roundings of 2^-24 of those."""
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    if not want.size or not np.abs(want).max():
        assert not np.abs(got).max(initial=0.0), what
        return
    d = got - want
    rel, big = np.linalg.norm(d) / np.linalg.norm(want), np.abs(d).max() / np.abs(want).max()
    more = (0.0, 0.0) if terms is None else (np.linalg.norm(terms) / np.linalg.norm(want),
                                             np.abs(terms).max() / np.abs(want).max())
    assert rel <= NORM[dtype] + 2.0 ** -21 * more[0] and big <= LARGEST[dtype] + 2.0 ** -21 * more[1], \
        f"{what}: norm {rel:.2e}, largest {big:.2e}"


def dx_terms(x, groups, dn, weight, eps, rms):
    """rstd (|du| + mean |du| + |u| mean |du u|), du = dn weight."""
    unit, inv, _ = gn._parts(x, groups, None, None, eps, rms)
    du = np.abs(dn * (1.0 if weight is None else weight)).reshape(x.shape[0], groups, -1)
    u = np.abs(unit).reshape(du.shape)
    return (inv * (du + du.mean(-1, keepdims=True) + u * (u * du).mean(-1, keepdims=True))).reshape(x.shape)


def close_sum(got, want, terms, rows, what):
    off = np.abs(f64(got) - want)
    assert (off <= (rows ** 0.5 * 2.0 ** -24 + 2.0 ** -21) * terms).all(), f"{what}: {(off / terms).max():.2e}"


def inputs(rows, groups, size, dtype, gated=True, affine=True):
    C = groups * size
    x = (torch.randn(rows, C, device="cuda") * torch.rand(C, device="cuda") + 0.3 * torch.randn(C, device="cuda"))
    kw = dict(gate=torch.randn(rows, C, device="cuda").to(DT[dtype]) if gated else None,
              weight=torch.randn(C, device="cuda") if affine else None,
              bias=torch.randn(C, device="cuda") if affine else None)
    return x.to(DT[dtype]), torch.randn(rows, C, device="cuda").to(DT[dtype]), kw


def check(rnn, x, groups, dy, kw, dtype, **opts):
    rows, C = x.shape
    ref = {n: f64(t) for n, t in kw.items()} | opts
    close(rnn.group_norm_forward(x, groups, **kw, **opts), gn.forward(f64(x), groups, **ref), dtype, "y")
    got = rnn.group_norm_backward(x, groups, dy, **kw, **opts)
    want = gn.backward(f64(x), groups, f64(dy), **ref)
    eps, rms, act = opts.get("eps", 1e-5), opts.get("rms", False), opts.get("activation", "silu")
    unit, inv, n = gn._parts(f64(x), groups, ref["weight"], ref["bias"], eps, rms)
    if kw["gate"] is not None:
        dn = np.abs(f64(dy) * gn._act(ref["gate"], act)[0])
    else:
        dn = np.abs(f64(dy)) * (1 if act == "none" else 1 + np.abs(n))
    close(got[0], want[0], dtype, "dx", dx_terms(f64(x), groups, dn, ref["weight"], eps, rms))
    if kw["gate"] is None:
        assert got[3] is None
    else:
        close(got[3], want[3], dtype, "dgate")
    if kw["weight"] is None:
        assert got[1] is None and got[2] is None
        return
    g = np.abs(f64(x)).reshape(rows, groups, -1)
    parts = (g + (0 if rms else np.abs(f64(x).reshape(g.shape).mean(-1, keepdims=True)))) * inv
    close_sum(got[1], want[1], (dn * parts.reshape(rows, C)).sum(0), rows, "dweight")
    close_sum(got[2], want[2], dn.sum(0), rows, "dbias")


SIZES = [1, 2, 3, 8, 10, 32, 50, 64, 80, 99, 128, 130, 192, 200, 256, 320, 512, 513, 1000, 1024]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(rnn, dtype, size):
    for rows, groups in ((1, 1), (5, 3), (37, 7)):
        x, dy, kw = inputs(rows, groups, size, dtype)
        check(rnn, x, groups, dy, kw, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_forms(rnn, dtype, rms, act, gated, affine):
    x, dy, kw = inputs(33, 5, 64, dtype, gated, affine)
    check(rnn, x, 5, dy, kw, dtype, activation=act, rms=rms, eps=1e-3)


@pytest.mark.parametrize("rows,groups,size", [(1023, 40, 64), (515, 32, 128), (2049, 4, 256), (300, 40, 99),
                                              (4099, 8, 50), (130, 16, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(rnn, dtype, rows, groups, size):
    """Several rows to a team, the last of them short."""
    x, dy, kw = inputs(rows, groups, size, dtype)
    check(rnn, x, groups, dy, kw, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_for_twice_the_workgroups(rnn, dtype):
    x, dy, kw = inputs(17001, 64, 8, dtype)
    check(rnn, x, 64, dy, kw, dtype)


def test_only_one_of_weight_and_bias(rnn):
    x, dy, kw = inputs(20, 3, 64, "f32")
    for n, i in (("weight", 1), ("bias", 2)):
        part = kw | {n: None}
        ref = {m: f64(t) for m, t in part.items()}
        close(rnn.group_norm_forward(x, 3, **part), gn.forward(f64(x), 3, **ref), "f32", "y")
        got, want = rnn.group_norm_backward(x, 3, dy, **part), gn.backward(f64(x), 3, f64(dy), **ref)
        close(got[0], want[0], "f32", "dx")
        assert got[i] is None
        np.testing.assert_allclose(f64(got[3 - i]), want[3 - i], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [0, 8, 7])
def test_strided_slices_of_a_joint_projection(rnn, dtype, first):
    """x and gate as slices, aligned to 16 bytes and not; the results are those of dense copies."""
    B, T, groups, size = 2, 9, 3, 64
    C = groups * size
    joint = torch.randn(B, T, 2 * C + 24 + first % 8, device="cuda").to(DT[dtype])
    x, z = joint[..., first:first + C], joint[..., first + C + 8:first + 2 * C + 8]
    w, b, dy = torch.randn(C, device="cuda"), torch.randn(C, device="cuda"), torch.randn(B, T, C, device="cuda").to(DT[dtype])
    kw = dict(weight=w, bias=b)
    y = rnn.group_norm_forward(x, groups, gate=z, **kw)
    want = rnn.group_norm_forward(x.contiguous(), groups, gate=z.contiguous(), **kw)
    grads = rnn.group_norm_backward(x, groups, dy, gate=z, **kw)
    plain = rnn.group_norm_backward(x.contiguous(), groups, dy, gate=z.contiguous(), **kw)
    ref = gn.forward(f64(x).reshape(-1, C), groups, weight=f64(w), bias=f64(b), gate=f64(z).reshape(-1, C))
    close(y.view(-1, C), ref, dtype, "y")
    if first != 7:
        assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(grads, plain))
    for p, q in zip((y, *grads), (want, *plain)):  # (another piece, another order of sums)
        close(p, f64(q), dtype if p.dim() == 3 else "f32", "dense copies")


def test_in_place(rnn):
    x, dy, kw = inputs(700, 8, 128, "bf16")
    y = rnn.group_norm_forward(x, 8, **kw)
    grads = rnn.group_norm_backward(x, 8, dy, **kw)
    x2, dy2 = x.clone(), dy.clone()
    got = rnn.group_norm_backward(x2, 8, dy2, dx=dy2, **kw)
    assert got[0] is dy2 and all(torch.equal(a, b) for a, b in zip(got, grads))
    assert rnn.group_norm_forward(x2, 8, y=x2, **kw) is x2 and torch.equal(x2, y)


def test_guards(rnn):
    """Nothing around the outputs is written."""
    for rows, groups, size in ((3, 3, 50), (5, 2, 64), (9, 1, 513)):
        C = groups * size
        x, dy, kw = inputs(rows, groups, size, "bf16")
        n = rows * C
        big = [torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        y, dx, dz = (t[32:32 + n].view(rows, C) for t in big)
        small = [torch.full((C + 64,), 7.0, device="cuda") for _ in range(2)]
        rnn.group_norm_forward(x, groups, y=y, **kw)
        rnn.group_norm_backward(x, groups, dy, dx=dx, dgate=dz, dweight=small[0][32:32 + C], dbias=small[1][32:32 + C], **kw)
        for t in big + small:
            assert (t[:32] == 7).all() and (t[-32:] == 7).all()
        assert torch.equal(y, rnn.group_norm_forward(x, groups, **kw))


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_what_is_not_finite_stays_in_its_row_and_group(rnn, value):
    x, dy, kw = inputs(40, 4, 64, "bf16")
    clean, grads = rnn.group_norm_forward(x, 4, **kw), rnn.group_norm_backward(x, 4, dy, **kw)
    x[11, 70] = float(value)
    y, got = rnn.group_norm_forward(x, 4, **kw), rnn.group_norm_backward(x, 4, dy, **kw)
    assert y[11, 64:128].isnan().all()
    for a, b in ((y, clean), (got[0], grads[0]), (got[3], grads[3])):
        a, b = a.clone(), b.clone()
        a[11, 64:128] = b[11, 64:128] = 0
        assert torch.equal(a, b)
    for a, b in zip(got[1:3], grads[1:3]):
        assert torch.equal(a[:64], b[:64]) and torch.equal(a[128:], b[128:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_gates_and_offsets(rnn, dtype):
    """Gates whose exponentials overflow, channels with an offset hundreds of times their spread."""
    x, dy, kw = inputs(16, 2, 128, dtype)
    x = (x.float() + 200.0).to(DT[dtype])
    kw["gate"][:, ::3] *= 100
    kw["gate"][0, :4] = torch.tensor([1e30, -1e30, 3e38, -3e38]).to(DT[dtype])
    kw["gate"][0, 4:6] = torch.tensor([60.0, -60.0])
    # (the difference to the mean is exact to 2^-24 of 200, 3e-5 of a spread of 0.5: float32 as it comes in)
    ref = {n: f64(t) for n, t in kw.items()}
    for act in ("silu", "sigmoid"):
        y = rnn.group_norm_forward(x, 2, activation=act, **kw)
        want = gn.forward(f64(x), 2, activation=act, **ref)
        assert y.isfinite().all() or not np.isfinite(want.astype(np.float32)).all()
        off, size = np.abs(f64(y) - want), np.abs(want)
        fine = np.isfinite(f64(y))
        spread = 200 * 2.0 ** -24 * 8  # of u, eight roundings at most
        bound = size * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -19) + spread * np.abs(ref["weight"]) * np.maximum(
            1, np.abs(ref["gate"])) / f64(x).reshape(16, 2, 128).std(-1).repeat(128, -1)
        assert (off[fine] <= bound[fine]).all()
        got = rnn.group_norm_backward(x, 2, dy, activation=act, **kw)
        assert not got[3][0, 1:6:2].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(rnn, dtype):
    x, dy, kw = inputs(0, 2, 64, dtype)
    assert rnn.group_norm_forward(x, 2, **kw).shape == (0, 128)
    dw = torch.full((128,), 7.0, device="cuda")
    got = rnn.group_norm_backward(x, 2, dy, dweight=dw, **kw)
    assert got[0].shape == (0, 128) and not dw.any() and not got[2].any()


def test_offsets_behind_32_bits(rnn):
    groups, size = 32, 128
    rows = 2 ** 31 // (groups * size) + 5
    x = torch.randn(rows, groups * size, device="cuda", dtype=torch.bfloat16)
    y = rnn.group_norm_forward(x, groups)
    dx, _, _, _ = rnn.group_norm_backward(x, groups, y)
    tail = slice(rows - 8, rows)
    want = rnn.group_norm_forward(x[tail].contiguous(), groups)
    assert torch.equal(y[tail], want)
    assert torch.equal(dx[tail], rnn.group_norm_backward(x[tail].contiguous(), groups, want)[0])


def test_other_stream_and_two_calls_at_once(rnn):
    data = [inputs(300, 8, 128, "bf16") for _ in range(2)]

    def step(i, **opts):
        x, dy, kw = data[i]
        return (rnn.group_norm_forward(x, 8, **kw, **opts), *rnn.group_norm_backward(x, 8, dy, **kw, **opts))

    want = [step(i) for i in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [step(i, stream=side[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


# ------------------------------------------------------------------------- the layer they make up

class Layer(torch.autograd.Function):
    """Linear attention over a batch, each head's readouts normalised and gated."""

    @staticmethod
    def forward(ctx, rnn, q, k, v, g, s0, weight, bias, gate):
        o, s = rnn.linear_attention_forward(q, k, v, g, s0)
        y = rnn.group_norm_forward(o.flatten(-2), v.shape[-2], weight=weight, bias=bias, gate=gate)
        ctx.rnn = rnn
        ctx.save_for_backward(q, k, v, g, s0, weight, bias, gate, o)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        q, k, v, g, s0, weight, bias, gate, o = ctx.saved_tensors
        rnn, heads = ctx.rnn, v.shape[-2]
        d_o, dw, db, dz = rnn.group_norm_backward(o.flatten(-2), heads, dy.contiguous(), weight=weight, bias=bias,
                                                  gate=gate)
        dq, dk, dv, dg, ds0 = rnn.linear_attention_backward(q, k, v, g, d_o.unflatten(-1, (heads, -1)), s0,
                                                            ds.contiguous())
        return None, dq, dk, dv, dg, ds0, dw, db, dz


def layer_inputs(B, T, Hk, Hv, K, V, dt):
    new = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    x = [new(B, T, Hk, K).to(dt), new(B, T, Hk, K).to(dt), new(B, T, Hv, V).to(dt), -torch.rand(Hv, device="cuda"),
         new(B, Hv, V, K), 1 + 0.1 * new(Hv * V), 0.1 * new(Hv * V), new(B, T, Hv * V).to(dt)]
    return x, new(B, T, Hv * V).to(dt), new(B, Hv, V, K)


def test_layer_gradients(rnn):
    """The whole layer in float32 against the oracles one after the other."""
    B, T, Hk, Hv, K, V = 1, 90, 1, 2, 64, 64
    x, dy, ds = layer_inputs(B, T, Hk, Hv, K, V, torch.float32)
    leaves = [t.clone().requires_grad_() for t in x]
    y, s = Layer.apply(rnn, *leaves)
    grads = torch.autograd.grad([y, s], leaves, [dy, ds])
    q, k, v, g, s0, w, b, z = (f64(t) for t in x)
    o, S, _ = la.forward(q[0], k[0], v[0], g, s0[0])
    o = o.reshape(T, -1)
    close(y[0], gn.forward(o, Hv, weight=w, bias=b, gate=z[0]), "f32", "y")
    close(s[0], S, "f32", "state")
    d_o, dw, db, dz = gn.backward(o, Hv, f64(dy[0]), weight=w, bias=b, gate=z[0])
    dq, dk, dv, dg, ds0 = la.backward(q[0], k[0], v[0], g, d_o.reshape(T, Hv, V), f64(ds[0]), s0[0])
    # sums through two operators, each within 1e-6 to 2e-6 of its own result; 1e-5 for those that cancel
    for n, a, want in zip(("q", "k", "v", "g", "s0", "w", "b", "z"), grads,
                          (dq[None], dk[None], dv[None], dg, ds0[None], dw, db, dz[None])):
        rel = np.linalg.norm(f64(a) - want) / np.linalg.norm(want)
        assert rel <= 1e-5, (n, rel)


def test_layer_captured_and_replayed(rnn):
    """A training step of the layer and a serving step behind it (prefill, then single tokens), captured and
    replayed with eager work in between, beside an eager graph of the same leaves."""
    B, T, Hk, Hv, K, V = 2, 130, 2, 4, 64, 128
    x, dy, ds = layer_inputs(B, T, Hk, Hv, K, V, torch.bfloat16)
    leaves = [t.clone().requires_grad_() for t in x]
    pool = torch.empty(B, Hv, V, K, device="cuda")
    outs = {}

    def work():
        y, s = Layer.apply(rnn, *leaves)
        outs["y"] = y.detach()
        for i, t in enumerate(torch.autograd.grad([y, s], leaves, [dy, ds])):
            outs[i] = t
        pool.copy_(s.detach())
        for t in range(3):
            o = rnn.linear_attention_decode(*(a[:, t].contiguous() for a in x[:3]), x[3], pool)
            outs[f"step{t}"] = rnn.group_norm_forward(o.flatten(-2), Hv, weight=x[5], bias=x[6], gate=x[7][:, t])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in outs.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    held = dict(outs)
    for _ in range(4):
        for t in held.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in held.items():
            assert torch.equal(t, want[n]), n
        rnn.group_norm_forward(x[7], Hv)  # eager work between the replays
        torch.cuda.synchronize()


def sigmoid_off(z, dtype):
    """How far the sigmoid may be off, relative to itself.  float: the exponential's 2^-23, the sum's and the
    quotient's 2^-24 each.  bf16: the hardware's exponential and reciprocal, 2^-23 each, and the sum's 2^-24; and the
    exponent, log2(e) z, is a float whose product and constant are off by 2^-24 and 2^-26 of it, of which 1 - s
    reaches the sigmoid (1.25 |z| 2^-24 log2(e) ln 2)."""
    s = 1 / (1 + np.exp(-z))
    return s, 2.0 ** -22 + 2.0 ** -24 + (1.25 * 2.0 ** -24 * np.abs(z) * (1 - s) if dtype == "bf16" else 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gradients_at_large_gates(rnn, dtype, act):
    """Value by value, channels whose gates are far out in every row (so that their dweight and dbias are sums of
    small terms only) beside ordinary ones; bounds from the roundings of each step."""
    rows, groups, size = 16, 2, 128
    x, dy, kw = inputs(rows, groups, size, dtype)
    far = [-100.0, -80.0, -60.0, -20.0, -8.0, 8.0, 12.0, 17.0, 20.0, 60.0, 80.0, 100.0]
    kw["gate"][:, 5:5 + len(far)] = torch.tensor(far).to(DT[dtype])
    kw["gate"][:, 200] *= 50
    ref = {n: f64(t) for n, t in kw.items()}
    y, (dx, dw, db, dz) = (rnn.group_norm_forward(x, groups, activation=act, **kw),
                           rnn.group_norm_backward(x, groups, dy, activation=act, **kw))
    want_y = gn.forward(f64(x), groups, activation=act, **ref)
    want = gn.backward(f64(x), groups, f64(dy), activation=act, **ref)

    X, D, z, w = f64(x), np.abs(f64(dy)), ref["gate"], np.abs(ref["weight"])
    unit, inv, n = gn._parts(X, groups, ref["weight"], ref["bias"], 1e-5, False)
    group = lambda t: t.reshape(rows, groups, size)  # noqa: E731
    flat = lambda t: t.reshape(rows, groups * size)  # noqa: E731
    mean = lambda t: np.broadcast_to(t.mean(-1, keepdims=True), t.shape)  # noqa: E731
    step, half = 2.0 ** -24, {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    u = np.abs(unit)
    # u: sums of 128 terms as trees (12 roundings), of the squares too (half of it in rstd), rsqrtf 2^-22, the
    # difference and the product: below 16 steps of |u| and of mean |x| rstd
    u_off = 16 * step * (u + flat(mean(group(np.abs(X))) * inv))
    n_off = w * u_off + 2 * step * (w * u + np.abs(n))
    s, rel = sigmoid_off(z, dtype)
    tiny = 2.0 ** -120  # the sigmoid's smallest normal values, times what it is multiplied with
    s_off = rel * s
    a, slope = gn._act(z, act)
    if act == "silu":
        a_off, slope_off = np.abs(z) * s_off + step * np.abs(a), (1 + np.abs(z)) * (s_off + 3 * step * s)
    else:
        a_off, slope_off = s_off, s_off + 3 * step * s
    a, slope = np.abs(a), np.abs(slope)
    off = {"y": a * n_off + np.abs(n) * a_off, "dgate": D * (slope * n_off + np.abs(n) * slope_off),
           "dbias": (D * a_off).sum(0) + (rows + 1) * step * (D * a).sum(0),
           "dweight": (D * (a_off * u + a * u_off)).sum(0) + (rows + 2) * step * (D * a * u).sum(0)}
    du, du_off = group(D * a * w), group(w * D * a_off + 2 * step * D * a * w)
    gu, gu_off = group(u), group(u_off)
    terms = du + mean(du) + gu * mean(du * gu)
    off["dx"] = flat(inv * (du_off + mean(du_off) + gu * mean(du_off * gu + du * gu_off) + gu_off * mean(du * gu)
                            + 32 * step * terms))
    for name, got, exact, kind in (("y", y, want_y, dtype), ("dgate", dz, want[3], dtype), ("dx", dx, want[0], dtype),
                                   ("dweight", dw, want[1], "f32"), ("dbias", db, want[2], "f32")):
        last = half if kind == dtype else step
        bound = off[name] * 1.01 + (last + 2 * step) * np.abs(exact) + tiny
        bad = np.abs(f64(got) - exact) / bound
        assert bad.max() <= 1, (name, bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    assert db[5 + far.index(-60.0)].abs() > 0 and (act == "silu" or db[5 + far.index(-80.0)].abs() > 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_outputs_at_the_largest_gates_are_finite_where_exact_ones_are(rnn, dtype, act):
    x, _, kw = inputs(16, 2, 128, dtype)
    ends = torch.tensor([1e30, -1e30, 3e38, -3e38, 200.0, -200.0, 89.0, -89.0]).to(DT[dtype])
    kw["gate"][:, 30:30 + len(ends)] = ends
    want = gn.forward(f64(x), 2, activation=act, **{n: f64(t) for n, t in kw.items()})
    fine = torch.from_numpy(want).to(DT[dtype]).isfinite().numpy()
    assert not fine.all() if act == "silu" else fine.all()
    y = rnn.group_norm_forward(x, 2, activation=act, **kw)
    assert np.array_equal(y.isfinite().cpu().numpy(), fine)
    close(torch.where(torch.from_numpy(fine).cuda() & (kw["gate"].abs() < 300), y, torch.zeros_like(y)),
          np.where(fine & (np.abs(f64(kw["gate"])) < 300), want, 0.0), dtype, "y")
