"""GPU parity of linear attention with its float64 implementation, at the lengths, layouts and masks
where it can go wrong.

Tolerances (2-norm of the difference over that of the result, unless stated):
 - float32, and the states from bf16 inputs, whose increments keep a float's 24 bits: sums of a few
   hundred terms in float32, 2^-24 each, sqrt(300) 2^-24 = 1e-6 for independent ones; 2e-6.
 - bf16 outputs: rounded once, off by at most 2^-8 = 3.9e-3; what they are the sums of is off by 2^-16
   per factor, far less: 4e-3 in the norm and of the largest.
 - dg adds products of either sign: per element of the state the sum over tokens of |D S|, independent
   between elements, each off by the errors of D and S, 2e-6 = 32 * 2^-24 of it.
"""
import ctypes

import numpy as np
import pytest

from oracle import linear_attention as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NORM = {"f32": 2e-6, "bf16": 4e-3}
LARGEST = {"f32": 1e-5, "bf16": 4e-3}
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
    torch.manual_seed(12)


def f64(x):
    return x.detach().to("cpu", torch.float64).numpy()


def close(got, want, dtype, what, terms=None):
    """``terms``: the same sums with the absolute values of all products."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    if not want.size or np.abs(want).max() < 2.0 ** -126:
        assert np.abs(got).max(initial=0.0) < 2.0 ** -125, what
        return
    d = got - want
    rel = np.linalg.norm(d) / np.linalg.norm(want)
    big = np.abs(d).max() / np.abs(want).max()
    # where products cancel (a single token's k . q is any number down to 0): the roundings of a sum of 64 or
    # 128 products, independent of each other, are off by sqrt(128) 2^-24 = 6.8e-7 of the sum of their sizes
    more = (0.0, 0.0) if terms is None else (np.linalg.norm(terms) / np.linalg.norm(want),
                                             np.abs(terms).max() / np.abs(want).max())
    assert rel <= NORM[dtype] + 6.8e-7 * more[0] and big <= LARGEST[dtype] + 6.8e-7 * more[1], \
        f"{what}: norm {rel:.2e}, largest {big:.2e}"


def inputs(total, Hk, Hv, K, V, dtype, seed, B=1):
    """q, k, v of a batch and the decays: heads that forget over one to some hundreds of tokens."""
    r = np.random.default_rng(seed)
    T = total // B
    x = [torch.from_numpy(r.normal(size=(B, T, H, C))).to(DT[dtype]).cuda() for H, C in ((Hk, K), (Hk, K), (Hv, V))]
    g = -np.exp2(-8 * r.random(Hv))
    return x + [torch.from_numpy(g.astype(np.float32)).cuda()]


def states(n, Hv, V, K, seed):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=(n, Hv, V, K)).astype(np.float32)).cuda()


def rows(x, B, a, b):
    return [f64(t[B, a:b]) for t in x[:3]] + [f64(x[3])]


def t32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def gate_scale(q, k, v, g, d_o, ds, s0):
    """Per head, what the terms of dg amount to: over the state's elements the 2-norm of the sum over
    tokens of |D S|."""
    T, Hk, K = k.shape
    Hv, V = v.shape[1:]
    _, _, trace = la.forward(q, k, v, g, s0)
    D = np.zeros((Hv, V, K)) if ds is None else np.array(ds)
    total, a = np.zeros((Hv, V, K)), np.exp(g)[:, None, None]
    for t in range(T - 1, -1, -1):
        D = a * (D + K ** -0.5 * d_o[t][:, :, None] * np.repeat(q[t], Hv // Hk, 0)[:, None, :])
        total += np.abs(D * trace[t])
    return np.sqrt((total ** 2).sum((1, 2)))


def check_gradients(grads, x, d_o, ds, s0, dtype, spans):
    """Against the formula's, sequence by sequence: spans of (row of the batch, first token, end)."""
    dg, spread = 0.0, 0.0
    for i, (b, lo, hi) in enumerate(spans):
        r, o = rows(x, b, lo, hi), f64(d_o[b, lo:hi])
        D, S = (None if t is None else f64(t[i]) for t in (ds, s0))
        ref = la.backward(*r, o, D, S)
        size = la.backward(*(np.abs(t) for t in r[:3]), r[3], np.abs(o), *(None if t is None else np.abs(t) for t in (D, S)))
        for n, a, want, terms in zip(("dq", "dk", "dv"), grads, ref, size):
            close(a[b, lo:hi], want, dtype, f"{n} of {i}", terms)
        close(grads[4][i], ref[4], "f32", f"ds0 of {i}")
        dg, spread = dg + ref[3], spread + gate_scale(*r, o, D, S)
    if grads[3] is not None:
        off = np.abs(f64(grads[3]) - dg)
        assert (off <= 32 * 2.0 ** -24 * spread + 2.0 ** -24 * np.abs(dg)).all(), (off, spread, dg)


# (dtype, K, V, Hk, Hv)
LAYOUTS = [("bf16", 64, 64, 1, 1), ("bf16", 64, 128, 2, 2), ("bf16", 128, 64, 1, 3), ("bf16", 128, 128, 2, 4),
           ("bf16", 128, 256, 1, 1), ("bf16", 64, 192, 1, 2), ("bf16", 128, 128, 3, 3), ("f32", 64, 64, 2, 4),
           ("f32", 64, 256, 1, 1), ("f32", 128, 128, 1, 2), ("f32", 128, 64, 1, 1), ("f32", 128, 128, 1, 1)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 129, 200])
def test_dense_forward(rnn, layout, T):
    dtype, K, V, Hk, Hv = layout
    B = 2
    x = inputs(B * T, Hk, Hv, K, V, dtype, 10 + T, B=B)
    s0 = states(B, Hv, V, K, T)
    o, s = rnn.linear_attention_forward(*x, s0=s0)
    for b in range(B):
        want, S, _ = la.forward(*rows(x, b, 0, T), f64(s0[b]))
        close(o[b], want, dtype, f"o[{b}]")
        close(s[b], S, "f32", "state")


@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3], LAYOUTS[5], LAYOUTS[7]], ids=str)
@pytest.mark.parametrize("long", [False, True])
def test_packed_forward_with_slots(rnn, layout, long):
    """Ragged lengths with empty ones, rows before and behind the sequences, states in a pool: kept,
    from zeros (-1, and out of range), dropped, forked from another slot."""
    dtype, K, V, Hk, Hv = layout
    lens = [700, 0, 64, 1, 513, 256, 0] if long else [5, 0, 64, 1, 130, 65, 0]
    first, behind = 3, 9
    cu = np.cumsum([first] + lens)
    total = cu[-1] + behind
    assert (rnn.linear_attention_forward_workspace_bytes(total, Hk, Hv, K, V, sequences=7, packed=True, dtype=dtype)
            > 0) == long
    x = inputs(total, Hk, Hv, K, V, dtype, 77)
    for t in x[:3]:  # what no sequence owns is not read
        t[0, :first] = float("nan")
        t[0, cu[-1]:] = float("nan")
    slots_in = [4, 2, -1, 7, 0, 11, 9]
    slots_out = [4, 2, 3, 7, -1, 6, 12]
    pool = states(10, Hv, V, K, 5)
    old = pool.clone()
    o = torch.full((1, total, Hv, V), 7.0, dtype=DT[dtype], device="cuda")
    rnn.linear_attention_forward(*x, s0=pool, s_out=pool, o=o, cu_seqlens=t32(cu), slots=t32(slots_out),
                                 slots_in=t32(slots_in))
    assert (o[0, :first] == 7).all() and (o[0, cu[-1]:] == 7).all()
    left = set(range(10))
    for i, n in enumerate(lens):
        a, b = cu[i], cu[i + 1]
        s0 = f64(old[slots_in[i]]) if 0 <= slots_in[i] < 10 else None
        want, S, _ = la.forward(*rows(x, 0, a, b), s0)
        close(o[0, a:b], want, dtype, f"o of sequence {i}")
        if 0 <= slots_out[i] < 10:
            left.discard(slots_out[i])
            close(pool[slots_out[i]], S, "f32", f"state of sequence {i}")
    for i in left:
        assert torch.equal(pool[i], old[i]), i


@pytest.mark.parametrize("layout", [LAYOUTS[1], LAYOUTS[3], LAYOUTS[4], LAYOUTS[9]], ids=str)
@pytest.mark.parametrize("T", [511, 1024, 1300])
def test_segments_against_float64(rnn, layout, T):
    dtype, K, V, Hk, Hv = layout
    assert rnn.linear_attention_forward_workspace_bytes(T, Hk, Hv, K, V, dtype=dtype) > 0
    x, s0, ds = inputs(T, Hk, Hv, K, V, dtype, T), states(1, Hv, V, K, 3), states(1, Hv, V, K, 4)
    x[3][0] = -0.0009  # still there after a thousand tokens
    start = s0.clone()
    o, s = rnn.linear_attention_forward(*x, s0=s0)
    want, S, _ = la.forward(*rows(x, 0, 0, T), f64(s0[0]))
    close(o[0], want, dtype, "o")
    close(s[0], S, "f32", "state")
    o2, s2 = rnn.linear_attention_forward(*x, s0=s0, s_out=s0)
    assert s2 is s0 and torch.equal(o, o2) and torch.equal(s, s2)
    d_o = torch.randn_like(o)
    grads = rnn.linear_attention_backward(*x, d_o, start, ds)
    check_gradients(grads, x, d_o, ds, start, dtype, [(0, 0, T)])
    fixed = rnn.linear_attention_backward(*x, d_o, start, ds, want_dg=False)
    assert fixed[3] is None
    for n, a, b in zip(("dq", "dk", "dv", "", "ds0"), grads, fixed):
        if n:
            close(a, f64(b), dtype, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V,started", [(64, 64, True), (64, 128, False), (128, 64, True)])
def test_a_few_segments_to_a_sequence(rnn, dtype, K, V, started):
    """Two or four in the forward, two in the backward, the last one shorter; from states and from none."""
    B, T, Hk, Hv = 3, 430, 2, 46
    x = inputs(B * T, Hk, Hv, K, V, dtype, 21, B)
    x[3][0], x[3][1] = 0.0, -1e-3
    s0, ds = (states(B, Hv, V, K, 3), states(B, Hv, V, K, 4)) if started else (None, None)
    o, s = rnn.linear_attention_forward(*x, s0=s0)
    for b in range(B):
        want, S, _ = la.forward(*rows(x, b, 0, T), None if s0 is None else f64(s0[b]))
        close(o[b], want, dtype, "o")
        close(s[b], S, "f32", "state")
    d_o = torch.from_numpy(np.random.default_rng(22).normal(size=(B, T, Hv, V))).to(DT[dtype]).cuda()
    grads = rnn.linear_attention_backward(*x, d_o, s0, ds)
    check_gradients(grads, x, d_o, ds, s0, dtype, [(b, 0, T) for b in range(B)])
    if started:  # in place: the starts lie where the ends are written
        pool, out = s0.clone(), ds.clone()
        o2, s2 = rnn.linear_attention_forward(*x, s0=pool, s_out=pool)
        close(o2, f64(o), dtype, "o in place")
        close(s2, f64(s), "f32", "state in place")
        for a, b, n in zip(rnn.linear_attention_backward(*x, d_o, s0, out, ds0=out), grads, ("dq", "dk", "dv", "", "ds0")):
            if n:
                close(a, f64(b), dtype, n)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("T", [1, 33, 64, 100, 150])
def test_gradients(rnn, layout, T):
    dtype, K, V, Hk, Hv = layout
    x = inputs(2 * T, Hk, Hv, K, V, dtype, 40 + T, B=2)
    s0, ds = states(2, Hv, V, K, 1), states(2, Hv, V, K, 2)
    d_o = torch.from_numpy(np.random.default_rng(9).normal(size=(2, T, Hv, V))).to(DT[dtype]).cuda()
    spans = [(0, 0, T), (1, 0, T)]
    check_gradients(rnn.linear_attention_backward(*x, d_o, s0, ds), x, d_o, ds, s0, dtype, spans)
    check_gradients(rnn.linear_attention_backward(*x, d_o, want_dg=False), x, d_o, None, None, dtype, spans)


def test_gradients_against_differences(rnn):
    """Float32: the directional derivative by central differences of the forward itself, and the
    gradients' product with the direction."""
    T, Hk, Hv, K, V = 70, 1, 2, 64, 64
    x, s0 = inputs(T, Hk, Hv, K, V, "f32", 50), states(1, Hv, V, K, 1)
    o, s = rnn.linear_attention_forward(*x, s0=s0)
    d_o, ds = torch.randn_like(o), torch.randn_like(s)
    grads = rnn.linear_attention_backward(*x, d_o, s0, ds)
    h = 2.0 ** -7
    for i, d in enumerate(grads):
        step = torch.randn_like(d) * (0.1 if i == 3 else 1.0)
        loss = []
        for sign in (h, -h):
            y = [t + sign * step if i == j else t for j, t in enumerate([*x, s0])]
            oo, ss = rnn.linear_attention_forward(*y[:4], s0=y[4])
            loss.append((oo.double() * d_o).sum() + (ss.double() * ds).sum())
        slope, want = float((loss[0] - loss[1]) / (2 * h)), float((d.double() * step).sum())
        # linear in q, k, v and s0 each, so that central differences are exact but for float32 sums: each
        # of N products of the loss is off by about 16 * 2^-24 of its size, which adds up as sqrt(N):
        # 1e-6 |o| |d_o| / h over two calls; in g the third derivative, (0.1 h)^2 / 6 T^2 of the slope, besides
        scale = float(o.double().norm() * 1.0 + s.double().norm())
        assert abs(slope - want) <= 1e-6 * scale / h + 2e-3 * abs(want), (i, slope, want, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_ragged_training_batch(rnn, dtype, long, shared):
    Hk, Hv, K, V = (1, 2, 64, 128) if shared else (2, 2, 128, 64)
    lens = [600, 0, 3, 257, 1, 512] if long else [64, 0, 3, 90, 1, 65]
    cu = np.cumsum([2] + lens)
    total = cu[-1] + 5
    x = inputs(total, Hk, Hv, K, V, dtype, 60)
    s0, ds = states(6, Hv, V, K, 1), states(6, Hv, V, K, 2)
    d_o = torch.randn(1, total, Hv, V, device="cuda").to(DT[dtype])
    clean = [t.clone() for t in x]
    for t in [*x[:3], d_o]:
        t[0, :2] = float("nan")
        t[0, cu[-1]:] = float("nan")
    out = [torch.full_like(t, 7.0) for t in x[:3]]
    # (a workspace of NaNs)
    work = torch.full((rnn.linear_attention_backward_workspace_bytes(total, Hk, Hv, K, V, sequences=6, packed=True,
                                                                     dtype=dtype),), 255, dtype=torch.uint8, device="cuda")
    grads = rnn.linear_attention_backward(*x, d_o, s0, ds, cu_seqlens=t32(cu), grads=out, workspace=work)
    check_gradients(grads, clean, d_o, ds, s0, dtype, [(0, cu[i], cu[i + 1]) for i in range(6)])
    for t in out:
        assert (t[0, :2] == 7).all() and (t[0, cu[-1]:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["forget", "lowest", "keep", "mixed"])
def test_extreme_decays(rnn, dtype, what):
    """Heads that forget everything at every token (-infinity, the type's lowest value) or nothing."""
    T, Hk, Hv, K, V = 150, 1, 2, 64, 64
    x = inputs(T, Hk, Hv, K, V, dtype, 21)
    x[3][:] = torch.tensor({"forget": [-float("inf")] * 2, "lowest": [torch.finfo(torch.float32).min, -1e30],
                            "keep": [0.0, -0.0], "mixed": [-float("inf"), 0.0]}[what])
    s0, ds, d_o = states(1, Hv, V, K, 1), states(1, Hv, V, K, 2), torch.randn(1, T, Hv, V, device="cuda").to(DT[dtype])
    o, s = rnn.linear_attention_forward(*x, s0=s0)
    want, S, _ = la.forward(*rows(x, 0, 0, T), f64(s0[0]))
    close(o[0], want, dtype, "o")
    close(s[0], S, "f32", "state")
    check_gradients(rnn.linear_attention_backward(*x, d_o, s0, ds), x, d_o, ds, s0, dtype, [(0, 0, T)])
    pool = s0.clone()
    one = [t[:, 0].contiguous() for t in x[:3]]
    od = rnn.linear_attention_decode(*one, x[3], pool)
    want, S, _ = la.forward(*rows(x, 0, 0, 1), f64(s0[0]))
    close(od, want, dtype, "decode")
    close(pool[0], S, "f32", "decoded state")


def test_slow_decays_over_many_chunks(rnn):
    """Decays close to one over 512 chunks, where a chunk's power rounded to a float would be off 512
    times in the same direction; against the same sums in float64 on the GPU, block by block."""
    T, K, V = 32768, 64, 64
    x = inputs(T, 4, 4, K, V, "bf16", 22)
    x[3][:] = -torch.tensor([2.0 ** -13, 3e-5, 1e-4, 7e-5])
    s0 = states(1, 4, V, K, 1)
    s = rnn.linear_attention_forward(*x, s0=s0)[1]
    q, k, v, g = (t.double() for t in x)
    S = s0[0].double()
    for a in range(0, T, 1024):
        w = torch.exp(g[:, None] * torch.arange(1023, -1, -1, device="cuda"))  # [H, 1024]
        S = torch.exp(1024 * g)[:, None, None] * S + torch.einsum("ht,thv,thk->hvk", w, v[0, a:a + 1024],
                                                                  k[0, a:a + 1024])
    close(s[0], f64(S), "f32", "state")
    # one chunk after the other, without segments: many heads of one long batch each
    pieces = [t[:, :8192].expand(64, -1, -1, -1).contiguous() for t in x[:3]]
    many = rnn.linear_attention_forward(*(t.repeat(1, 1, 4, 1) for t in pieces), x[3].repeat(4))[1]
    S = torch.zeros_like(S)
    for a in range(0, 8192, 1024):
        w = torch.exp(g[:, None] * torch.arange(1023, -1, -1, device="cuda"))
        S = torch.exp(1024 * g)[:, None, None] * S + torch.einsum("ht,thv,thk->hvk", w, v[0, a:a + 1024],
                                                                  k[0, a:a + 1024])
    close(many[63, 12:], f64(S), "f32", "state of whole sequences")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs_of_a_joint_projection(rnn, dtype):
    B, T, Hk, Hv, K, V = 2, 70, 2, 4, 64, 128
    x = inputs(B * T, Hk, Hv, K, V, dtype, 3, B=B)
    joint = torch.cat([t.flatten(2) for t in x[:3]], -1)
    q, k, v = joint.split([Hk * K, Hk * K, Hv * V], -1)
    views = (q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (Hv, V)))
    o, s = rnn.linear_attention_forward(*x)
    o2, s2 = rnn.linear_attention_forward(*views, x[3])
    assert torch.equal(o, o2) and torch.equal(s, s2)
    d_o = torch.randn_like(o)
    want = rnn.linear_attention_backward(*x, d_o)
    got = rnn.linear_attention_backward(*views, x[3], d_o)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool, pool2 = states(B, Hv, V, K, 1), states(B, Hv, V, K, 1)
    a = rnn.linear_attention_decode(*(t[:, 5].contiguous() for t in x[:3]), x[3], pool)
    b = rnn.linear_attention_decode(*(t[:, 5] for t in views), x[3], pool2)
    assert torch.equal(a, b) and torch.equal(pool, pool2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_strides(rnn, dtype):
    """2^23 elements from token to token: a chunk's rows lie over 2 GiB."""
    T, Hk, Hv, K, V = 67, 1, 2, 64, 64
    x = inputs(T, Hk, Hv, K, V, dtype, 31)
    wide = torch.empty(T, 1 << 23, device="cuda", dtype=DT[dtype])
    parts, at = [], (1 << 23) - 64 * 4
    for t, n in zip(x[:3], (64, 64, 128)):
        parts.append(wide[:, at:at + n].view(1, T, n // 64, 64))
        parts[-1].copy_(t)
        at += n
    d_o = torch.from_numpy(np.random.default_rng(32).normal(size=(1, T, Hv, V))).to(DT[dtype]).cuda()
    for a, b in zip(rnn.linear_attention_forward(*parts, x[3]), rnn.linear_attention_forward(*x)):
        assert torch.equal(a, b)
    for a, b in zip(rnn.linear_attention_backward(*parts, x[3], d_o), rnn.linear_attention_backward(*x, d_o)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["q", "k", "v", "g"])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_what_is_not_finite_stays_in_its_heads_and_behind_its_chunk(rnn, name, value):
    B, T, Hk, Hv, K, V = 2, 200, 2, 4, 64, 64
    x = inputs(B * T, Hk, Hv, K, V, "bf16", 8, B=B)
    clean, clean_s = rnn.linear_attention_forward(*x)
    if name == "g":
        x[3][1] = float("nan")
        hit, rest = [1], [0, 1]
    else:
        x["qkv".index(name)][0, 140, 1].view(-1)[0] = float(value)
        hit, rest = [2, 3] if name in "qk" else [1], [0]
    o, s = rnn.linear_attention_forward(*x)
    keep = [h for h in range(Hv) if h not in hit]
    for b in range(B):
        if b not in rest:
            assert torch.equal(o[b], clean[b]) and torch.equal(s[b], clean_s[b])
        assert torch.equal(o[b][:, keep], clean[b][:, keep]) and torch.equal(s[b][keep], clean_s[b][keep])
    if name != "g":
        assert torch.equal(o[0, :128][:, hit], clean[0, :128][:, hit])
    assert not o[0, 140][hit].isfinite().all()
    if name != "q":
        assert not any(s[0, h].isfinite().all() for h in hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_batches(rnn, dtype):
    s0 = states(3, 2, 64, 64, 4)
    for x, cu in ((inputs(0, 1, 2, 64, 64, dtype, 1, B=3), None),
                  (inputs(0, 1, 2, 64, 64, dtype, 1), torch.zeros(4, dtype=torch.int32, device="cuda"))):
        o, s = rnn.linear_attention_forward(*x, s0=s0, cu_seqlens=cu)
        assert o.numel() == 0 and torch.equal(s, s0)
        o, s = rnn.linear_attention_forward(*x, cu_seqlens=cu) if cu is None else (o, s)
        dg = torch.full((2,), 7.0, device="cuda")
        grads = rnn.linear_attention_backward(*x, o, s0, ds_T=s0, cu_seqlens=cu, dg=dg)
        assert torch.equal(grads[4], s0) and not dg.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 70), (2, 64), (3, 5)])
def test_many_heads_of_one_key_head_over_few_tokens(rnn, dtype, B, T):
    """More heads than chunks: what is summed over heads stays within the tokens."""
    x = inputs(B * T, 1, 64, 64, 64, dtype, 12, B)
    d_o = torch.from_numpy(np.random.default_rng(13).normal(size=(B, T, 64, 64))).to(DT[dtype]).cuda()
    room = [torch.full((B * T + 4096, *t.shape[2:]), 7.0, dtype=DT[dtype], device="cuda") for t in x[:3]]
    grads = [t[2048:2048 + B * T].view(B, T, *t.shape[1:]) for t in room]
    got = rnn.linear_attention_backward(*x, d_o, grads=grads)
    check_gradients(got, x, d_o, None, None, dtype, [(b, 0, T) for b in range(B)])
    for t in room:
        assert (t[:2048] == 7).all() and (t[2048 + B * T:] == 7).all()


def test_gradient_of_the_state_in_place(rnn):
    for T in (100, 700):
        x, ds = inputs(T, 1, 2, 64, 128, "bf16", 5), states(1, 2, 128, 64, 6)
        d_o = torch.randn(1, T, 2, 128, device="cuda").bfloat16()
        want = rnn.linear_attention_backward(*x, d_o, None, ds)
        got = rnn.linear_attention_backward(*x, d_o, None, ds, ds0=ds)
        assert got[4] is ds and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("B", [1, 7])
def test_decode(rnn, layout, B):
    """Single tokens one after the other against the float64 recurrence; with slots, padded rows
    (a slot outside the pool) and the other states stay as they are."""
    dtype, K, V, Hk, Hv = layout
    steps = 3
    x = inputs(B * steps, Hk, Hv, K, V, dtype, 70, B=B)
    pool = states(B + 3, Hv, V, K, 3)
    old = pool.clone()
    slots = torch.randperm(B + 3)[:B].int()
    if B > 2:
        slots[1], slots[2] = -1, B + 3
    slots = slots.cuda()
    plain = old[slots.long().clamp(0, B + 2)].contiguous()
    os = []
    for t in range(steps):
        one = [a[:, t].contiguous() for a in x[:3]]
        o = torch.full((B, Hv, V), 7.0, dtype=DT[dtype], device="cuda")
        os.append(rnn.linear_attention_decode(*one, x[3], pool, slots=slots, o=o))
        o2 = rnn.linear_attention_decode(*one, x[3], plain)
        live = [b for b in range(B) if 0 <= slots[b] < B + 3]
        assert torch.equal(os[-1][live], o2[live])
    touched = []
    for b in range(B):
        if not 0 <= slots[b] < B + 3:
            assert all((o[b] == 7).all() for o in os)
            continue
        touched.append(int(slots[b]))
        want, S, _ = la.forward(*rows(x, b, 0, steps), f64(old[slots[b]]))
        close(torch.stack([o[b] for o in os]), want, dtype, "o")
        close(pool[slots[b]], S, "f32", "state")
    for i in range(B + 3):
        assert i in touched or torch.equal(pool[i], old[i])


def test_prefill_then_decode_is_one_sequence(rnn):
    """A prompt in two pieces and single tokens after it, through a pool, against one pass."""
    T, Hk, Hv, K, V = 140, 2, 4, 128, 128
    x = inputs(T, Hk, Hv, K, V, "bf16", 80)
    pool = torch.zeros(4, Hv, V, K, device="cuda")
    slot, fresh = t32([2]), t32([-1])
    pool[2] = 5.0  # of an earlier sequence
    os = []
    for a, b, start in ((0, 70, fresh), (70, 135, slot)):
        piece = [t[:, a:b].contiguous() for t in x[:3]]
        os.append(rnn.linear_attention_forward(*piece, x[3], s0=pool, s_out=pool, slots=slot, slots_in=start)[0][0])
    for t in range(135, T):
        os.append(rnn.linear_attention_decode(*(a[:, t].contiguous() for a in x[:3]), x[3], pool, slots=slot))
    want, S, _ = la.forward(*rows(x, 0, 0, T))
    close(torch.cat(os), want, "bf16", "o")
    close(pool[2], S, "f32", "state")
    assert not pool[[0, 1, 3]].any()


def test_other_stream_and_two_calls_at_once(rnn):
    T, Hk, Hv, K, V = 600, 2, 4, 128, 128
    xs = [inputs(T, Hk, Hv, K, V, "bf16", 90 + i) for i in range(2)]
    d_o = torch.randn(1, T, Hv, V, device="cuda").bfloat16()

    def step(x, **kw):
        return (*rnn.linear_attention_forward(*x, **kw), *rnn.linear_attention_backward(*x, d_o, **kw))

    want = [step(x) for x in xs]
    side = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [step(x, stream=s) for x, s in zip(xs, side)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    with torch.cuda.stream(side[0]):
        got = step(xs[0])
    side[0].synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))


@pytest.mark.parametrize("T", [200, 900])
def test_graph_replays_equal_the_eager_run(rnn, T):
    """Prefill, a fork of its states, a decode step of all and a training step, captured together and
    replayed with eager work in between."""
    Hk, Hv, K, V = 1, 2, 64, 64
    cu = t32([0, 70, 71, T])
    x = inputs(T, Hk, Hv, K, V, "bf16", 95)
    one = [a[0, :6].contiguous() for a in x[:3]]
    slots, src, dst, six = t32([0, 1, 2]), t32([0, 1, 2]), t32([5, 4, 3]), t32([0, 1, 2, 3, 4, 5])
    start = states(6, Hv, V, K, 1)
    pool = start.clone()
    d_o = torch.randn(1, T, Hv, V, device="cuda").bfloat16()
    outs = {}

    def work():
        pool.copy_(start)
        outs["o"], _ = rnn.linear_attention_forward(*x, s0=pool, s_out=pool, slots=slots, cu_seqlens=cu)
        rnn.state_move(pool, src, dst)
        outs["d"] = rnn.linear_attention_decode(*one, x[3], pool, slots=six)
        outs["g"] = torch.cat([t.flatten().float() for t in rnn.linear_attention_backward(*x, d_o, cu_seqlens=cu)])

    work()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in outs.items()} | {"pool": pool.clone()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    held = dict(outs)
    for _ in range(4):
        for t in held.values():
            t.zero_()
        pool.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in held.items():
            assert torch.equal(t, want[n]), n
        assert torch.equal(pool, want["pool"])
        rnn.linear_attention_forward(*x)  # eager work between the replays
        torch.cuda.synchronize()


def test_wrong_offsets_stay_inside_the_buffers(rnn):
    """cu_seqlens that decrease, are negative or pass the end give no access outside (the rows
    around the buffers keep their guard values)."""
    Hk, Hv, K, V = 1, 1, 64, 64
    for n in (100, 1000):
        x = inputs(n, Hk, Hv, K, V, "bf16", 97)
        big = torch.full((1, n + 40, Hv, V), 7.0, dtype=torch.bfloat16, device="cuda")
        o = big[:, 20:n + 20]
        s = states(4, Hv, V, K, 1)
        for cu in ([0, n // 2, 30, 2 * n, n], [-5, 10, 1 << 30, -(1 << 31), n], [n, 0, n, 0, n]):
            rnn.linear_attention_forward(*x, s0=s, o=o, cu_seqlens=t32(cu))
            rnn.linear_attention_backward(*x, x[2].clone(), s, cu_seqlens=t32(cu),
                                          grads=(torch.empty_like(x[0]), torch.empty_like(x[1]), o))
            torch.cuda.synchronize()
            assert (big[:, :20] == 7).all() and (big[:, n + 20:] == 7).all()


def test_results_do_not_depend_on_the_batch_or_the_run(rnn):
    Hk, Hv, K, V = 2, 4, 128, 128
    x = inputs(4 * 130, Hk, Hv, K, V, "bf16", 98, B=4)
    d_o = torch.randn(4, 130, Hv, V, device="cuda").bfloat16()

    def step(y, d):
        o, s = rnn.linear_attention_forward(*y)
        return (o, s, *rnn.linear_attention_backward(*y, d))

    a, b = step(x, d_o), step(x, d_o)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    if rnn.linear_attention_forward_workspace_bytes(520, Hk, Hv, K, V, sequences=4):
        return
    alone = step([t[2:3].contiguous() for t in x[:3]] + [x[3]], d_o[2:3].contiguous())
    for i, (p, q) in enumerate(zip(a, alone)):
        assert i == 5 or torch.equal(p[2:3], q), i


def test_offsets_behind_32_bits(rnn):
    """A pool of 2.1e9 elements: prefill and decode at its end.  Then a batch whose values lie behind 2^31
    elements, training included."""
    Hk, Hv, K, V = 1, 8, 128, 128
    slots = 2 ** 31 // (Hv * V * K) + 3
    pool = torch.empty(slots, Hv, V, K, device="cuda")
    last = t32([slots - 1])
    start = states(1, Hv, V, K, 1)
    pool[-1] = start[0]
    x = inputs(70, Hk, Hv, K, V, "bf16", 99)
    o, s = rnn.linear_attention_forward(*x, s0=start)
    op, _ = rnn.linear_attention_forward(*x, s0=pool, s_out=pool, slots=last)
    assert torch.equal(o, op) and torch.equal(s[0], pool[-1])
    one = [a[:, 0].contiguous() for a in x[:3]]
    a = rnn.linear_attention_decode(*one, x[3], s)
    b = rnn.linear_attention_decode(*one, x[3], pool, slots=last)
    assert torch.equal(a, b) and torch.equal(s[0], pool[-1])
    del pool

    Hk, Hv, K, V = 1, 64, 64, 128
    T, short = 2 ** 31 // (Hv * V) + 64, 70
    total = T + short
    gen = torch.Generator("cuda").manual_seed(3)
    new = lambda *shape: torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=gen)  # noqa: E731
    x = [new(1, total, Hk, K), new(1, total, Hk, K), new(1, total, Hv, V), -torch.rand(Hv, device="cuda")]
    cu = t32([0, T, total])
    d_o = new(1, total, Hv, V)
    o, s = rnn.linear_attention_forward(*x, cu_seqlens=cu)
    grads = rnn.linear_attention_backward(*x, d_o, cu_seqlens=cu)
    tail = [t[:, T:].contiguous() for t in x[:3]] + [x[3]]
    to, ts = rnn.linear_attention_forward(*tail)
    want = rnn.linear_attention_backward(*tail, d_o[:, T:].contiguous())
    close(o[:, T:], f64(to), "bf16", "o")
    close(s[1], f64(ts[0]), "f32", "state")
    for name, a, b in zip(("dq", "dk", "dv"), grads, want):
        close(a[:, T:], f64(b), "bf16", name)
    close(grads[4][1], f64(want[4][0]), "f32", "ds0")


@pytest.mark.parametrize("n,K,V", [(4096, 64, 64), (2048, 64, 256)])
def test_large_batches(rnn, n, K, V):
    """Prefill, gradients and single tokens of more sequences and heads than 2^18 - 1, against the same in two
    halves (whole sequences, so bit for bit) and, for some, against float64."""
    T, H = 2, 64
    gen = torch.Generator("cuda").manual_seed(n)
    new = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    x = [new(n, T, H, C).bfloat16() for C in (K, K, V)] + [-torch.rand(H, device="cuda", generator=gen)]
    s0, d_o, ds = new(n, H, V, K), new(n, T, H, V).bfloat16(), new(n, H, V, K)
    halves = [slice(0, n // 2), slice(n // 2, n)]
    part = lambda h: [t[h] for t in x[:3]] + [x[3]]  # noqa: E731
    some = (0, n // 2, n - 1)

    o, s = rnn.linear_attention_forward(*x, s0=s0)
    for h in halves:
        a, b = rnn.linear_attention_forward(*part(h), s0=s0[h])
        assert torch.equal(o[h], a) and torch.equal(s[h], b)
    for i in some:
        want, S, _ = la.forward(*rows(x, i, 0, T), f64(s0[i]))
        close(o[i], want, "bf16", "o")
        close(s[i], S, "f32", "state")

    one, pool = [t[:, 0].contiguous() for t in x[:3]], s0.clone()
    od = rnn.linear_attention_decode(*one, x[3], pool)
    for i in some:
        want, S, _ = la.forward(*rows(x, i, 0, 1), f64(s0[i]))
        close(od[i:i + 1], want, "bf16", "decode")
        close(pool[i], S, "f32", "decoded state")
    for h in halves:
        again = s0[h].clone()
        assert torch.equal(od[h], rnn.linear_attention_decode(*(t[h] for t in one), x[3], again))
        assert torch.equal(pool[h], again)
    del s, pool, again, a, b

    grads = rnn.linear_attention_backward(*x, d_o, s0, ds)
    dg = []
    for h in halves:
        got = rnn.linear_attention_backward(*part(h), d_o[h], s0[h], ds[h])
        for name, a, b in zip(("dq", "dk", "dv", "", "ds0"), grads, got):
            assert not name or torch.equal(a[h], b), name
        dg.append(got[3].double())
    # sums in float64, each rounded once to float32
    bound = 2.0 ** -24 * (grads[3].abs() + dg[0].abs() + dg[1].abs()) * 1.01
    assert ((dg[0] + dg[1] - grads[3]).abs() <= bound).all()
    picked = [tuple(t[i:i + 1] for i in some) for t in (grads[0], grads[1], grads[2], grads[4])]
    for j, i in enumerate(some):
        got = (*(t[j] for t in picked[:3]), None, picked[3][j])
        check_gradients(got, [t[i:i + 1] for t in x[:3]] + [x[3]], d_o[i:i + 1], ds[i:i + 1], s0[i:i + 1], "bf16",
                        [(0, 0, T)])


def launches(call):
    """Kernels that the call enqueues: the nodes of a graph that it is captured into."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    count = ctypes.c_size_t()
    nodes = ctypes.CDLL("libamdhip64.so").hipGraphGetNodes
    assert nodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(count)) == 0
    return count.value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_without_the_final_states_are_launched_together(rnn, dtype):
    """No cotangent of the final states and no gradient of the first ones: nothing is in another's place, and
    the launches and results are those of zeros; only ds0 in ds_T's place takes one more launch."""
    T, H, K, V = 100, 2, 64, 64
    x = inputs(T, H, H, K, V, dtype, 14)
    d_o = torch.from_numpy(np.random.default_rng(15).normal(size=(1, T, H, V))).to(DT[dtype]).cuda()
    zeros, ds0 = torch.zeros(1, H, V, K, device="cuda"), torch.empty(1, H, V, K, device="cuda")
    without = lambda: rnn.linear_attention_backward(*x, d_o, want_ds0=False)  # noqa: E731
    apart = lambda: rnn.linear_attention_backward(*x, d_o, None, zeros, ds0=ds0)  # noqa: E731
    for a, b in zip(without()[:4], apart()):
        assert torch.equal(a, b)
    same = ds0.clone()
    same.zero_()
    in_place = lambda: rnn.linear_attention_backward(*x, d_o, None, same, ds0=same)  # noqa: E731
    in_place()
    assert torch.equal(same, ds0)
    assert launches(without) == launches(apart) < launches(in_place)


def backward_segments(rnn, T, H, K, V, dtype):
    """Segments that the gradients of one dense sequence are computed in, from the workspace's size (a state and
    a cotangent of each, and 8 bytes for dg)."""
    size = rnn.linear_attention_backward_workspace_bytes(T, H, H, K, V, dtype=dtype)
    one = H * (2 * V * K * 4 + 8)
    return size // one if size % one == 0 else 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("T,H,count", [(193, 1, 4), (250, 3, 4), (450, 40, 4), (270, 64, 3), (384, 50, 3)])
@pytest.mark.parametrize("started", [True, False])
def test_three_and_four_segments_joined_in_the_backward(rnn, dtype, K, V, T, H, count, started):
    """Of one and two chunks, the last one short or whole; heads that keep nearly everything, and others."""
    assert backward_segments(rnn, T, H, K, V, dtype) == count
    x = inputs(T, H, H, K, V, dtype, 16 + T)
    x[3][0] = -1e-3
    if H > 1:
        x[3][1] = 0.0
    s0, ds = (states(1, H, V, K, 3), states(1, H, V, K, 4)) if started else (None, None)
    d_o = torch.from_numpy(np.random.default_rng(17).normal(size=(1, T, H, V))).to(DT[dtype]).cuda()
    grads = rnn.linear_attention_backward(*x, d_o, s0, ds)
    some = sorted({0, min(1, H - 1), H - 1})
    of = lambda t: None if t is None else t[:, some]  # noqa: E731
    picked = [t[:, :, some] for t in grads[:3]] + [grads[3][some], of(grads[4])]
    check_gradients(picked, [t[:, :, some] for t in x[:3]] + [x[3][some]], d_o[:, :, some], of(ds), of(s0), dtype,
                    [(0, 0, T)])
    fixed = rnn.linear_attention_backward(*x, d_o, s0, ds, want_dg=False)
    assert fixed[3] is None
    for a, b, n in zip(fixed, grads, ("dq", "dk", "dv", "", "ds0")):
        if n:  # (dq takes the state in two parts where dg is not wanted, else in three)
            close(a, f64(b), dtype, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,count", [(700, 60, 2), (500, 40, 3), (1100, 30, 4)])
def test_joined_segments_with_slots(rnn, dtype, T, H, count):
    """Dense sequences from one pool into another, whose entries are in another order; one starts from zeros."""
    B, K, V = 2, 64, 128
    size = rnn.linear_attention_forward_workspace_bytes(B * T, H, H, K, V, sequences=B, dtype=dtype)
    assert size == count * B * H * V * K * 4
    x = inputs(B * T, H, H, K, V, dtype, 18, B)
    x[3][0], x[3][1] = 0.0, -1e-3
    pool, out = states(4, H, V, K, 5), torch.full((4, H, V, K), 7.0, device="cuda")
    o, _ = rnn.linear_attention_forward(*x, s0=pool, s_out=out, slots=t32([3, 0]), slots_in=t32([1, -1]))
    some = [0, 1, H - 1]
    for b, (start, end) in enumerate(((1, 3), (None, 0))):
        r = rows([t[:, :, some] for t in x[:3]] + [x[3][some]], b, 0, T)
        want, S, _ = la.forward(*r, None if start is None else f64(pool[start][some]))
        close(o[b][:, some], want, dtype, "o")
        close(out[end][some], S, "f32", "state")
    assert (out[1:3] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_prompt_among_single_tokens(rnn, dtype):
    """A serving step's batch of one prompt and nine sequences that go on by a token (and an empty one), through a
    pool and with gradients: right, and the same bits each time."""
    Hk, Hv, K, V = 16, 32, 64, 64
    lens = [1, 1, 1, 1100, 1, 0, 1, 1, 1, 1, 1]
    n, cu = len(lens), np.cumsum([0] + lens)
    x = inputs(cu[-1], Hk, Hv, K, V, dtype, 19)
    x[3][0] = -1e-3
    start, ds = states(n + 3, Hv, V, K, 6), states(n, Hv, V, K, 7)
    slots = list(np.random.default_rng(20).permutation(n + 3)[:n])
    d_o = torch.from_numpy(np.random.default_rng(21).normal(size=(1, cu[-1], Hv, V))).to(DT[dtype]).cuda()
    first = None
    for _ in range(3):
        pool = start.clone()
        o, _ = rnn.linear_attention_forward(*x, s0=pool, s_out=pool, slots=t32(slots), cu_seqlens=t32(cu))
        s0 = start[slots].contiguous()
        got = (o, pool, *rnn.linear_attention_backward(*x, d_o, s0, ds, cu_seqlens=t32(cu)))
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    # key heads 0 and 15, with the value heads that read them
    ks, vs = [0, Hk - 1], [0, 1, Hv - 2, Hv - 1]
    y = [x[0][:, :, ks], x[1][:, :, ks], x[2][:, :, vs], x[3][vs]]
    for i in range(n):
        want, S, _ = la.forward(*rows(y, 0, cu[i], cu[i + 1]), f64(s0[i][vs]))
        close(o[0, cu[i]:cu[i + 1]][:, vs], want, dtype, f"o of {i}")
        close(pool[slots[i]][vs], S, "f32", f"state of {i}")
    for i in set(range(n + 3)) - set(slots):
        assert torch.equal(pool[i], start[i])
    grads = [got[2][:, :, ks], got[3][:, :, ks], got[4][:, :, vs], got[5][vs], got[6][:, vs]]
    check_gradients(grads, y, d_o[:, :, vs], ds[:, vs], s0[:, vs], dtype, [(0, cu[i], cu[i + 1]) for i in range(n)])


@pytest.mark.parametrize("name", ["q", "k", "v", "d_o"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_what_is_not_finite_stay_in_their_heads(rnn, dtype, name):
    """And dq at and behind its chunk, dk and dv at and before it, their chunks counted from the end."""
    B, T, Hk, Hv, K, V, at = 2, 180, 2, 4, 64, 64, 100
    x = inputs(B * T, Hk, Hv, K, V, dtype, 23, B=B)
    s0, ds = states(B, Hv, V, K, 1), states(B, Hv, V, K, 2)
    d_o = torch.from_numpy(np.random.default_rng(24).normal(size=(B, T, Hv, V))).to(DT[dtype]).cuda()
    clean = rnn.linear_attention_backward(*x, d_o, s0, ds)
    (d_o if name == "d_o" else x["qkv".index(name)])[0, at, 1, 5] = float("nan")
    key, hit = (1, [2, 3]) if name in "qk" else (0, [1])
    keep = [h for h in range(Hv) if h not in hit]
    got = rnn.linear_attention_backward(*x, d_o, s0, ds)
    dq, dk, dv, dg, ds0 = zip(got, clean)
    for a, b in (dq, dk, dv, ds0):
        assert torch.equal(a[1], b[1])
    for a, b in (dq, dk):
        assert torch.equal(a[0][:, 1 - key], b[0][:, 1 - key])
    assert torch.equal(dv[0][0][:, keep], dv[1][0][:, keep])
    assert torch.equal(dg[0][keep], dg[1][keep]) and torch.equal(ds0[0][0][keep], ds0[1][0][keep])
    assert torch.equal(dq[0][0, :64], dq[1][0, :64])
    for a, b in (dk, dv):
        assert torch.equal(a[0, T - 64:], b[0, T - 64:])
    assert not all(dg[0][hit].isfinite())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [90, 400])  # whole, and in segments
def test_growing_states(rnn, dtype, T):
    """Log decays above 0 are computed as they stand."""
    Hk, Hv, K, V = 1, 2, 64, 64
    x = inputs(T, Hk, Hv, K, V, dtype, 25)
    x[3][:] = torch.tensor([0.03, 1e-3])
    s0, ds = states(1, Hv, V, K, 1), states(1, Hv, V, K, 2)
    d_o = torch.from_numpy(np.random.default_rng(26).normal(size=(1, T, Hv, V))).to(DT[dtype]).cuda()
    o, s = rnn.linear_attention_forward(*x, s0=s0)
    want, S, _ = la.forward(*rows(x, 0, 0, T), f64(s0[0]))
    for h in range(Hv):  # (the one that grows a thousandfold would hide the other)
        close(o[0][:, h], want[:, h], dtype, "o")
        close(s[0, h], S[h], "f32", "state")
    check_gradients(rnn.linear_attention_backward(*x, d_o, s0, ds), x, d_o, ds, s0, dtype, [(0, 0, T)])
    one, pool = [t[:, 0].contiguous() for t in x[:3]], s0.clone()
    od = rnn.linear_attention_decode(*one, x[3], pool)
    want, S, _ = la.forward(*rows(x, 0, 0, 1), f64(s0[0]))
    close(od, want, dtype, "decode")
    close(pool[0], S, "f32", "decoded state")
