"""GPU parity of the gated delta rule with its float64 implementation, at the lengths,
layouts and masks where it can go wrong.

Tolerances (2-norm of the difference over that of the result, unless stated):
 - float32: sums of a few hundred terms in float32, 2^-24 each; 2e-6.
 - float32 states from bf16 inputs: operands split into two bf16 parts, off by at most 2^-17 of the
   value, in four products one after the other (S k, T R, U k^T and the cotangents'): 4 * 2^-17 = 2^-15.
 - bf16 outputs: a rounding is off by at most 2^-8, 2^-8 / sqrt(3) = 2.3e-3 in the mean over a binade's
   worst case.  o takes S, U, P and itself rounded: sqrt(4) * 2.3e-3 = 4.5e-3; the gradients S, D, U, dR, M
   and themselves: sqrt(6) * 2.3e-3 = 5.6e-3.  1e-2 for both leaves a factor below two for correlation.
   Single elements: 2^-8 of themselves and 6 * 2^-8 of the largest for the operands: 7 * 2^-8 < 3e-2 of
   the largest.
"""
import numpy as np
import pytest

from oracle import gated_delta as gd

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NORM = {"f32": 2e-6, "bf16": 1e-2}
LARGEST = {"f32": 1e-5, "bf16": 3e-2}
STATE = {"f32": 2e-6, "bf16": 2.0 ** -15}
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
    torch.manual_seed(11)


def f64(x):
    return x.detach().to("cpu", torch.float64).numpy()


def close(got, want, dtype, what, norm=NORM, largest=LARGEST):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    if not want.size or np.abs(want).max() < 2.0 ** -126:
        assert np.abs(got).max(initial=0.0) < 2.0 ** -125, what
        return
    d = got - want
    d[np.abs(d) < 2.0 ** -126] = 0  # below the smallest normal float32 there is nothing to be right about
    rel = np.linalg.norm(d) / np.linalg.norm(want)
    big = np.abs(d).max() / np.abs(want).max()
    assert rel <= norm[dtype] and big <= largest[dtype], f"{what}: norm {rel:.2e}, largest {big:.2e}"


def close_state(got, want, dtype, what="state"):
    close(got, want, dtype, what, STATE, {"f32": 1e-5, "bf16": 2.0 ** -15})


def inputs(total, Hk, Hv, K, V, dtype, seed, B=1, unit=False, slow=False):
    r = np.random.default_rng(seed)
    T = total // B
    x = dict(q=r.normal(size=(B, T, Hk, K)), k=r.normal(size=(B, T, Hk, K)), v=r.normal(size=(B, T, Hv, V)),
             g=-np.log1p(np.exp(r.normal(size=(B, T, Hv)))) * (0.01 if slow else 1.0) ** r.random((B, T, Hv)),
             beta=1 / (1 + np.exp(-r.normal(size=(B, T, Hv)))))
    if unit:
        for n in "qk":
            x[n] /= np.linalg.norm(x[n], axis=-1, keepdims=True)
    return {n: torch.from_numpy(a).to(DT[dtype]).cuda() for n, a in x.items()}


def states(n, Hv, V, K, seed):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=(n, Hv, V, K)).astype(np.float32)).cuda()


NAMES = ("q", "k", "v", "g", "beta")


def rows(x, B, a, b):
    return [f64(x[n][B, a:b]) for n in NAMES]


# (dtype, K, V, Hk, Hv, normalize)
LAYOUTS = [("bf16", 64, 64, 1, 1, False), ("bf16", 64, 128, 2, 2, True), ("bf16", 128, 64, 1, 3, True),
           ("bf16", 128, 128, 2, 4, True), ("bf16", 128, 256, 1, 1, False), ("f32", 64, 64, 2, 4, True),
           ("f32", 64, 256, 1, 1, True), ("f32", 128, 128, 1, 2, False), ("f32", 128, 64, 1, 1, True)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 129, 200])
def test_dense_forward(rnn, layout, T):
    dtype, K, V, Hk, Hv, normalize = layout
    B = 2
    x = inputs(B * T, Hk, Hv, K, V, dtype, 10 + T, B=B, unit=not normalize)
    s0 = states(B, Hv, V, K, T)
    o, s = rnn.gated_delta_forward(*x.values(), s0=s0, normalize=normalize)
    for b in range(B):
        want, S, _ = gd.forward(*rows(x, b, 0, T), f64(s0[b]), normalize=normalize)
        close(o[b], want, dtype, f"o[{b}]")
        close_state(s[b], S, dtype)


@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3], LAYOUTS[5]], ids=str)
def test_packed_forward_with_slots(rnn, layout):
    """Ragged lengths with empty ones, rows before and behind the sequences, states in a pool: kept,
    from zeros (-1, and out of range), dropped, forked from another slot."""
    dtype, K, V, Hk, Hv, normalize = layout
    lens = [5, 0, 64, 1, 130, 65, 0]
    first, behind = 3, 9
    cu = np.cumsum([first] + lens)
    total = cu[-1] + behind
    x = inputs(total, Hk, Hv, K, V, dtype, 77, unit=not normalize)
    for n in NAMES:  # what no sequence owns is not read
        x[n][0, :first] = float("nan")
        x[n][0, cu[-1]:] = float("nan")
    slots_in = [4, 2, -1, 7, 0, 11, 9]
    slots_out = [4, 2, 3, 7, -1, 6, 12]
    pool = states(10, Hv, V, K, 5)
    old = pool.clone()
    o = torch.full((1, total, Hv, V), 7.0, dtype=DT[dtype], device="cuda")
    t32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    rnn.gated_delta_forward(*x.values(), s0=pool, s_out=pool, o=o, cu_seqlens=t32(cu), slots=t32(slots_out),
                            slots_in=t32(slots_in), normalize=normalize)
    assert (o[0, :first] == 7).all() and (o[0, cu[-1]:] == 7).all()
    left = set(range(10))
    for i, n in enumerate(lens):
        a, b = cu[i], cu[i + 1]
        s0 = f64(old[slots_in[i]]) if 0 <= slots_in[i] < 10 else None
        want, S, _ = gd.forward(*rows(x, 0, a, b), s0, normalize=normalize)
        close(o[0, a:b], want, dtype, f"o of sequence {i}")
        if 0 <= slots_out[i] < 10:
            left.discard(slots_out[i])
            close_state(pool[slots_out[i]], S, dtype, f"state of sequence {i}")
    for i in left:
        assert torch.equal(pool[i], old[i]), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs_of_a_joint_projection(rnn, dtype):
    B, T, Hk, Hv, K, V = 2, 70, 2, 4, 64, 128
    x = inputs(B * T, Hk, Hv, K, V, dtype, 3, B=B)
    joint = torch.cat([x["q"].flatten(2), x["k"].flatten(2), x["v"].flatten(2)], -1)
    q, k, v = joint.split([Hk * K, Hk * K, Hv * V], -1)
    views = (q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (Hv, V)))
    o, s = rnn.gated_delta_forward(*x.values(), normalize=True)
    o2, s2 = rnn.gated_delta_forward(*views, x["g"], x["beta"], normalize=True)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    d_o = torch.randn_like(o)
    _, _, ck, u = rnn.gated_delta_forward_train(*x.values(), normalize=True)
    want = rnn.gated_delta_backward(*x.values(), d_o, ck, u, normalize=True)
    got = rnn.gated_delta_backward(*views, x["g"], x["beta"], d_o, ck, u, normalize=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool, pool2 = states(B, Hv, V, K, 1), states(B, Hv, V, K, 1)
    one = [t[:, 5] for t in x.values()]
    a = rnn.gated_delta_decode(*(t.contiguous() for t in one), pool)
    b = rnn.gated_delta_decode(*(t[:, 5] for t in views), *(t.contiguous() for t in one[3:]), pool2)
    assert torch.equal(a, b) and torch.equal(pool, pool2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["forget", "lowest", "keep", "silent", "reflect", "repeat", "strong"])
def test_extreme_gates_and_keys(rnn, dtype, what):
    """Decays that forget everything (-infinity, the type's lowest value) or nothing, write strengths
    of 0 and 2, equal keys, and strong decays whose sums over a chunk reach thousands."""
    B, T, Hk, Hv, K, V = 1, 150, 1, 2, 64, 64
    x = inputs(T, Hk, Hv, K, V, dtype, 21)
    if what in ("forget", "lowest"):
        x["g"][0, [0, 3, 40, 64, 65, 127, 128]] = -float("inf") if what == "forget" else torch.finfo(DT[dtype]).min
    elif what == "keep":
        x["g"].zero_()
    elif what == "silent":
        x["beta"].zero_()
    elif what == "reflect":
        x["beta"].fill_(2.0)
    elif what == "repeat":
        x["k"][:] = x["k"][:, :1].clone()
        x["beta"].fill_(1.0)
    elif what == "strong":
        x["g"][0, ::3] = -90.0
    s0, ds, d_o = states(1, Hv, V, K, 1), states(1, Hv, V, K, 2), torch.randn(B, T, Hv, V, device="cuda").to(DT[dtype])
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, normalize=True)
    want, S, _ = gd.forward(*rows(x, 0, 0, T), f64(s0[0]), normalize=True)
    close(o[0], want, dtype, "o")
    close_state(s[0], S, dtype)
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, normalize=True)
    ref = gd.backward(*rows(x, 0, 0, T), f64(d_o[0]), f64(ds[0]), f64(s0[0]), normalize=True)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
        if n == "dg" and what == "repeat":
            # with one key for all tokens and beta = 1 the terms of dg cancel (each token replaces what the
            # one before it wrote), so the bound is on the terms: in bf16 each is a product of at most two
            # vectors rounded to bf16 (2^-8 of every product of elements for each), in float32 a sum of 64
            # or 128 products (2^-24 each), and the sum is rounded once
            terms = decay_terms(*rows(x, 0, 0, T), f64(d_o[0]), f64(s0[0]), f64(ds[0]))
            unit, last = (2 * 2.0 ** -8 * 1.01, 2.0 ** -8) if dtype == "bf16" else (128 * 2.0 ** -24, 2.0 ** -24)
            assert (np.abs(f64(a[0]) - b) <= unit * terms + last * np.abs(b)).all()
        else:
            close(a[0], b, dtype, n)
    close_state(grads[5][0], ref[5], dtype, "ds0")


def decay_terms(q, k, v, g, beta, d_o, s0, ds):
    """The sums of dg over chunks of 64 tokens with the absolute value of every product of elements."""
    q, k, scale, T = gd._unit(q), gd._unit(k), q.shape[-1] ** -0.5, len(q)
    _, _, trace = gd.forward(q, k, v, g, beta, s0)
    dR = gd.backward(q, k, v, g, beta, d_o, ds, s0)[2] / beta[..., None]
    out = np.zeros_like(g)
    for a in range(0, T, 64):
        z = slice(a, min(T, a + 64))
        D = gd.backward(q[z.stop:], k[z.stop:], v[z.stop:], g[z.stop:], beta[z.stop:], d_o[z.stop:], ds,
                        trace[z.stop])[5] if z.stop < T else ds
        for h in range(g.shape[1]):
            j = h // (g.shape[1] // k.shape[1])
            S, qq, kk, be = trace[a][h], q[z, j], k[z, j], beta[z, h]
            U = np.stack([be[i] * (v[a + i, h] - np.exp(g[a + i, h]) * trace[a + i][h] @ kk[i])
                          for i in range(len(kk))])
            G = np.cumsum(g[z, h])
            E = np.exp(np.minimum(G[:, None] - G[None], 0))
            o_, r_, u_ = np.abs(d_o[z, h]), np.abs(dR[z, h]), np.abs(U)
            M = E * (scale * np.abs(qq @ kk.T) * (o_ @ u_.T) + be[:, None] * np.abs(kk @ kk.T) * (r_ @ u_.T))
            entry = np.exp(G) * (scale * (o_ * (np.abs(qq) @ np.abs(S).T)).sum(-1)
                                 + be * (r_ * (np.abs(kk) @ np.abs(S).T)).sum(-1))
            leave = np.exp(G[-1] - G) * (u_ * (np.abs(kk) @ np.abs(D[h]).T)).sum(-1)
            whole = np.exp(G[-1]) * (np.abs(D[h]) * np.abs(S)).sum()
            for t in range(len(kk)):
                out[a + t, h] = M[t:, :t].sum() + entry[t:].sum() + leave[:t].sum() + whole
    return out


@pytest.mark.parametrize("name", NAMES)
def test_a_nan_stays_in_its_sequence_and_behind_its_chunk(rnn, name):
    B, T, Hk, Hv, K, V = 2, 200, 2, 4, 64, 64
    x = inputs(B * T, Hk, Hv, K, V, "bf16", 8, B=B)
    clean, clean_s = rnn.gated_delta_forward(*x.values(), normalize=True)
    x[name][0, 140, 1].view(-1)[0] = float("nan")
    o, s = rnn.gated_delta_forward(*x.values(), normalize=True)
    hit = [2, 3] if name in "qk" else [1]
    keep = [h for h in range(Hv) if h not in hit]
    assert torch.equal(o[1], clean[1]) and torch.equal(s[1], clean_s[1])
    assert torch.equal(o[0][:, keep], clean[0][:, keep]) and torch.equal(s[0][keep], clean_s[0][keep])
    assert torch.equal(o[0, :128][:, hit], clean[0, :128][:, hit])
    assert o[0, 140][hit].isnan().any()
    if name != "q":
        assert all(s[0, h].isnan().any() for h in hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_batches(rnn, dtype):
    s0 = states(3, 2, 64, 64, 4)
    x = inputs(0, 1, 2, 64, 64, dtype, 1, B=3)
    o, s = rnn.gated_delta_forward(*x.values(), s0=s0)
    assert o.numel() == 0 and torch.equal(s, s0)
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values())
    assert ck.shape[0] == 0 and not s.any()
    assert torch.equal(rnn.gated_delta_backward(*x.values(), o, ck, u, ds_T=s0)[5], s0)
    x = inputs(0, 1, 2, 64, 64, dtype, 1)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, cu_seqlens=cu)
    assert torch.equal(s, s0)
    assert torch.equal(rnn.gated_delta_backward(*x.values(), o, ck, u, ds_T=s0, cu_seqlens=cu)[5], s0)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("T", [1, 33, 64, 100, 150])
def test_gradients(rnn, layout, T):
    dtype, K, V, Hk, Hv, normalize = layout
    x = inputs(T, Hk, Hv, K, V, dtype, 40 + T, unit=not normalize, slow=True)
    s0, ds = states(1, Hv, V, K, 1), states(1, Hv, V, K, 2)
    d_o = torch.from_numpy(np.random.default_rng(9).normal(size=(1, T, Hv, V))).to(DT[dtype]).cuda()
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, normalize=normalize)
    plain = rnn.gated_delta_forward(*x.values(), s0=s0, normalize=normalize)
    assert torch.equal(o, plain[0]) and torch.equal(s, plain[1])
    _, _, trace = gd.forward(*rows(x, 0, 0, T), f64(s0[0]), normalize=normalize)
    for c in range(ck.shape[0]):
        close(ck[c], trace[64 * c], dtype, f"state {c}")
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, normalize=normalize)
    ref = gd.backward(*rows(x, 0, 0, T), f64(d_o[0]), f64(ds[0]), f64(s0[0]), normalize=normalize)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
        close(a[0], b, dtype, n)
    close_state(grads[5][0], ref[5], dtype, "ds0")


def test_gradients_against_differences(rnn):
    """Float32: the directional derivative by central differences of the forward itself, and the
    gradients' product with the direction."""
    T, Hk, Hv, K, V = 70, 1, 2, 64, 64
    x = inputs(T, Hk, Hv, K, V, "f32", 50, slow=True)
    s0 = states(1, Hv, V, K, 1)
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, normalize=True)
    d_o, ds = torch.randn_like(o), torch.randn_like(s)
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, normalize=True)
    h = 2.0 ** -7
    for i, d in enumerate(grads):
        step = torch.randn_like(d)
        loss = []
        for sign in (h, -h):
            y = [t + sign * step if i == j else t for j, t in enumerate([*x.values(), s0])]
            oo, ss = rnn.gated_delta_forward(*y[:5], s0=y[5], normalize=True)
            loss.append((oo.double() * d_o).sum() + (ss.double() * ds).sum())
        slope, want = float((loss[0] - loss[1]) / (2 * h)), float((d.double() * step).sum())
        # the differences: h^2 = 6e-5 of the third derivative along the step (normed steps of size about h,
        # a few times the slope's scale), float32 noise 1e-7 |loss| / h far below; the scale is the product
        # of the two norms over the square root of the dimension, the size of a random product
        scale = float(d.norm() * step.norm()) / d.numel() ** 0.5
        assert abs(slope - want) <= 2e-3 * scale, (i, slope, want, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_training_batch(rnn, dtype):
    Hk, Hv, K, V = 1, 2, 64, 64
    lens = [64, 0, 3, 90, 1]
    cu = np.cumsum([2] + lens)
    total = cu[-1] + 5
    x = inputs(total, Hk, Hv, K, V, dtype, 60)
    s0, ds = states(5, Hv, V, K, 1), states(5, Hv, V, K, 2)
    d_o = torch.randn(1, total, Hv, V, device="cuda").to(DT[dtype])
    for t in [*x.values(), d_o]:
        t[0, :2] = float("nan")
        t[0, cu[-1]:] = float("nan")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, cu_seqlens=cut, normalize=True)
    out = [torch.full_like(t, 7.0) for t in x.values()]
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, cu_seqlens=cut, normalize=True, grads=out)
    for i in range(5):
        a, b = cu[i], cu[i + 1]
        want, S, trace = gd.forward(*rows(x, 0, a, b), f64(s0[i]), normalize=True)
        ref = gd.backward(*rows(x, 0, a, b), f64(d_o[0, a:b]), f64(ds[i]), f64(s0[i]), normalize=True)
        close(o[0, a:b], want, dtype, "o")
        close_state(s[i], S, dtype)
        for n, got, r in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
            close(got[0, a:b], r, dtype, f"{n} of sequence {i}")
        close_state(grads[5][i], ref[5], dtype, "ds0")
    for t in out:
        assert (t[0, :2] == 7).all() and (t[0, cu[-1]:] == 7).all()


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("B", [1, 7])
def test_decode(rnn, layout, B):
    """Single tokens one after the other against the float64 recurrence; with slots, padded rows
    (a slot outside the pool) and the other states stay as they are."""
    dtype, K, V, Hk, Hv, normalize = layout
    steps = 3
    x = inputs(B * steps, Hk, Hv, K, V, dtype, 70, B=B, unit=not normalize)
    pool = states(B + 3, Hv, V, K, 3)
    old = pool.clone()
    slots = torch.randperm(B + 3)[:B].int()
    if B > 2:
        slots[1], slots[2] = -1, B + 3
    slots = slots.cuda()
    plain = old[slots.long().clamp(0, B + 2)].contiguous()
    os = []
    for t in range(steps):
        one = [a[:, t].contiguous() for a in x.values()]
        o = torch.full((B, Hv, V), 7.0, dtype=DT[dtype], device="cuda")
        os.append(rnn.gated_delta_decode(*one, pool, slots=slots, normalize=normalize, o=o))
        o2 = rnn.gated_delta_decode(*one, plain, normalize=normalize)
        live = [b for b in range(B) if 0 <= slots[b] < B + 3]
        assert torch.equal(os[-1][live], o2[live])
    touched = []
    for b in range(B):
        if not 0 <= slots[b] < B + 3:
            assert all((o[b] == 7).all() for o in os)
            continue
        touched.append(int(slots[b]))
        want, S, _ = gd.forward(*rows(x, b, 0, steps), f64(old[slots[b]]), normalize=normalize)
        close(torch.stack([o[b] for o in os]), want, dtype, "o")
        close_state(pool[slots[b]], S, "f32")
    for i in range(B + 3):
        assert i in touched or torch.equal(pool[i], old[i])


def test_decode_forgets_at_minus_infinity(rnn):
    x = [a[:, 0].contiguous() for a in inputs(2, 1, 1, 64, 64, "bf16", 1, B=2).values()]
    x[3][0] = -float("inf")
    pool = states(2, 1, 64, 64, 1)
    o = rnn.gated_delta_decode(*x, pool)
    want, S, _ = gd.forward(*(f64(a[0])[None] for a in x), np.zeros((1, 64, 64)))
    close(o[:1], want, "bf16", "o")
    close_state(pool[0], S, "f32")


def test_prefill_then_decode_is_one_sequence(rnn):
    """A prompt in two pieces and single tokens after it, through a pool, against one pass."""
    T, Hk, Hv, K, V = 140, 2, 4, 128, 128
    x = inputs(T, Hk, Hv, K, V, "bf16", 80)
    pool = torch.zeros(4, Hv, V, K, device="cuda")
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([-1], dtype=torch.int32, device="cuda")
    pool[2] = 5.0  # of an earlier sequence
    os = []
    for a, b, start in ((0, 70, fresh), (70, 135, slot)):
        piece = [t[:, a:b].contiguous() for t in x.values()]
        os.append(rnn.gated_delta_forward(*piece, s0=pool, s_out=pool, slots=slot, slots_in=start,
                                          normalize=True)[0][0])
    for t in range(135, T):
        os.append(rnn.gated_delta_decode(*(a[:, t].contiguous() for a in x.values()), pool, slots=slot,
                                         normalize=True))
    want, S, _ = gd.forward(*rows(x, 0, 0, T), normalize=True)
    close(torch.cat(os), want, "bf16", "o")
    close_state(pool[2], S, "bf16")
    assert not pool[[0, 1, 3]].any()


def test_other_stream_and_two_calls_at_once(rnn):
    T, Hk, Hv, K, V = 300, 2, 4, 128, 128
    xs = [inputs(T, Hk, Hv, K, V, "bf16", 90 + i) for i in range(2)]
    want = [rnn.gated_delta_forward(*x.values(), normalize=True) for x in xs]
    side = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [rnn.gated_delta_forward(*x.values(), normalize=True, stream=s) for x, s in zip(xs, side)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with torch.cuda.stream(side[0]):
        o, s = rnn.gated_delta_forward(*xs[0].values(), normalize=True)
    side[0].synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(s, want[0][1])


def test_graph_replays_equal_the_eager_run(rnn):
    """Prefill, a fork of its states, a decode step of all and a training step, captured together and
    replayed with eager work in between."""
    Hk, Hv, K, V = 1, 2, 64, 64
    cu = torch.tensor([0, 70, 71, 200], dtype=torch.int32, device="cuda")
    x = inputs(200, Hk, Hv, K, V, "bf16", 95)
    one = [a[0, :6].contiguous() for a in x.values()]
    t32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, src, dst, six = t32([0, 1, 2]), t32([0, 1, 2]), t32([5, 4, 3]), t32([0, 1, 2, 3, 4, 5])
    start = states(6, Hv, V, K, 1)
    pool = start.clone()
    d_o = torch.randn(1, 200, Hv, V, device="cuda").bfloat16()
    outs = {}

    def work():
        pool.copy_(start)
        outs["o"], _ = rnn.gated_delta_forward(*x.values(), s0=pool, s_out=pool, slots=slots, cu_seqlens=cu,
                                               normalize=True)
        rnn.state_move(pool, src, dst)
        outs["d"] = rnn.gated_delta_decode(*one, pool, slots=six, normalize=True)
        _, _, ck, u = rnn.gated_delta_forward_train(*x.values(), cu_seqlens=cu, normalize=True)
        outs["g"] = torch.cat([t.flatten().float() for t in rnn.gated_delta_backward(
            *x.values(), d_o, ck, u, cu_seqlens=cu, normalize=True)])

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
        rnn.gated_delta_forward(*x.values(), normalize=True)  # eager work between the replays
        torch.cuda.synchronize()


def test_wrong_offsets_stay_inside_the_buffers(rnn):
    """cu_seqlens that decrease, are negative or pass the end give no access outside (the rows
    around the buffers keep their guard values)."""
    Hk, Hv, K, V = 1, 1, 64, 64
    x = inputs(100, Hk, Hv, K, V, "bf16", 97)
    big = torch.full((1, 140, Hv, V), 7.0, dtype=torch.bfloat16, device="cuda")
    o = big[:, 20:120]
    s = states(4, Hv, V, K, 1)
    for cu in ([0, 50, 30, 200, 100], [-5, 10, 1 << 30, -(1 << 31), 100], [100, 0, 100, 0, 100]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        rnn.gated_delta_forward(*x.values(), s0=s, o=o, cu_seqlens=c, normalize=True)
        torch.cuda.synchronize()
        assert (big[:, :20] == 7).all() and (big[:, 120:] == 7).all()


def test_results_do_not_depend_on_the_batch_or_the_run(rnn):
    Hk, Hv, K, V = 2, 4, 128, 128
    x = inputs(4 * 130, Hk, Hv, K, V, "bf16", 98, B=4)
    d_o = torch.randn(4, 130, Hv, V, device="cuda").bfloat16()

    def step(y, d):
        o, s, ck, u = rnn.gated_delta_forward_train(*y, normalize=True)
        return (o, s, *rnn.gated_delta_backward(*y, d, ck, u, normalize=True))

    a, b = step([*x.values()], d_o), step([*x.values()], d_o)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    alone = step([t[2:3].contiguous() for t in x.values()], d_o[2:3].contiguous())
    assert all(torch.equal(p[2:3], q) for p, q in zip(a, alone))


@pytest.mark.parametrize("layout", [("bf16", 64, 64, 1, 2), ("bf16", 64, 128, 2, 2), ("bf16", 128, 128, 1, 2),
                                    ("bf16", 128, 64, 1, 1), ("bf16", 128, 256, 1, 1), ("f32", 64, 64, 1, 2),
                                    ("f32", 128, 256, 1, 1), ("f32", 128, 128, 2, 2)], ids=str)
def test_long_sequences_of_few_heads(rnn, layout):
    """Sequences long enough to be done in parallel segments, in place, next to short ones, against
    the same tokens in pieces that are too short for it (the state carried in float32)."""
    dtype, K, V, Hk, Hv = layout
    lens = [3000, 1100, 0, 1500, 5]
    x = inputs(sum(lens), Hk, Hv, K, V, dtype, 33, slow=True)
    x["g"] *= 0.05                                      # far memories
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    pool = states(5, Hv, V, K, 3)
    old = pool.clone()
    need = rnn.gated_delta_forward_workspace_bytes
    # the segments' states and transitions need workspace besides that of the chunks
    assert need(sum(lens), Hk, Hv, K, V, sequences=5, packed=True, dtype=dtype) > \
        need(64, 1, 1, K, V, dtype=dtype) * Hv * (sum(lens) // 64 + 5)
    o, s = rnn.gated_delta_forward(*x.values(), s0=pool, s_out=pool, cu_seqlens=cu, normalize=True)
    ot, st, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=old, cu_seqlens=cu, normalize=True)
    assert torch.equal(o, ot) and torch.equal(s, st)
    for i, n in enumerate(lens):
        a, S, parts = int(cu[i]), old[i:i + 1].clone(), []
        for b in range(a, a + n, 400):
            piece = [t[:, b:min(b + 400, a + n)].contiguous() for t in x.values()]
            one, S = rnn.gated_delta_forward(*piece, s0=S, normalize=True)
            parts.append(one)
        close_state(pool[i], f64(S[0]), dtype)
        if n:
            close(o[:, a:a + n], f64(torch.cat(parts, 1)), dtype, f"o of sequence {i}")


# (dtype, K, V, Hk, Hv)
@pytest.mark.parametrize("layout", [("bf16", 64, 128, 1, 2), ("bf16", 128, 128, 1, 2), ("bf16", 128, 256, 1, 3),
                                    ("bf16", 64, 64, 2, 2), ("f32", 64, 64, 1, 3), ("f32", 128, 128, 1, 2)], ids=str)
def test_many_ragged_sequences(rnn, layout):
    """More sequences than CUs, whose states lie in a pool in another order: the workgroups of the most
    waves, and one workgroup for all value heads of a key head.  Every tenth sequence against float64."""
    dtype, K, V, Hk, Hv = layout
    n = 300
    r = np.random.default_rng(5)
    lens = r.integers(0, 150, n)
    lens[[0, 10, 20, 30, 40]] = [0, 1, 64, 149, 128]
    cu, total = np.cumsum([0, *lens]), int(lens.sum())
    x = inputs(total, Hk, Hv, K, V, dtype, 71)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    order = r.permutation(n + 4)[:n]
    old = states(n + 4, Hv, V, K, 6)
    pool = old.clone()
    o, _ = rnn.gated_delta_forward(*x.values(), s0=pool, s_out=pool, cu_seqlens=cut, normalize=True,
                                   slots=torch.tensor(order, dtype=torch.int32, device="cuda"))
    s0 = old[torch.from_numpy(order).cuda()].contiguous()
    ot, st, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, cu_seqlens=cut, normalize=True)
    d_o, ds = torch.randn(1, total, Hv, V, device="cuda").to(DT[dtype]), states(n, Hv, V, K, 7)
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, cu_seqlens=cut, normalize=True)
    spare = sorted(set(range(n + 4)) - set(order.tolist()))
    assert torch.equal(pool[spare], old[spare])
    for i in range(0, n, 10):
        a, b = cu[i], cu[i + 1]
        want, S, _ = gd.forward(*rows(x, 0, a, b), f64(s0[i]), normalize=True)
        ref = gd.backward(*rows(x, 0, a, b), f64(d_o[0, a:b]), f64(ds[i]), f64(s0[i]), normalize=True)
        for y, z in ((o, pool[order[i]]), (ot, st[i])):
            close(y[0, a:b], want, dtype, f"o of sequence {i}")
            close_state(z, S, dtype, f"state of sequence {i}")
        for name, got, w in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
            close(got[0, a:b], w, dtype, f"{name} of sequence {i}")
        close_state(grads[5][i], ref[5], dtype, f"ds0 of sequence {i}")


@pytest.mark.parametrize("layout", [("bf16", 64, 128, 1, 1), ("bf16", 128, 128, 1, 2), ("f32", 64, 64, 1, 2),
                                    ("f32", 128, 128, 1, 1)], ids=str)
@pytest.mark.parametrize("T", [1024, 1087, 2049])
def test_segments_against_float64(rnn, layout, T):
    """One sequence that is done in segments, whole and as the second of a graph's two replays."""
    dtype, K, V, Hk, Hv = layout
    x = inputs(T, Hk, Hv, K, V, dtype, 80 + T, slow=True)
    s0 = states(1, Hv, V, K, 8)
    need = rnn.gated_delta_forward_workspace_bytes
    # more workspace than the chunks need
    assert need(T, Hk, Hv, K, V, dtype=dtype) > need(64, 1, 1, K, V, dtype=dtype) * Hv * ((T + 63) // 64)
    o, s = rnn.gated_delta_forward(*x.values(), s0=s0, normalize=True)
    want, S, _ = gd.forward(*rows(x, 0, 0, T), f64(s0[0]), normalize=True)
    close(o[0], want, dtype, "o")
    close_state(s[0], S, dtype)
    work = torch.empty(need(T, Hk, Hv, K, V, dtype=dtype), dtype=torch.uint8, device="cuda")
    o2, s2 = torch.empty_like(o), torch.empty_like(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rnn.gated_delta_forward(*x.values(), s0=s0, normalize=True, o=o2, s_out=s2, workspace=work)
    for _ in range(3):
        work.fill_(255)  # what a call finds in its workspace does not matter (NaN here)
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(s, s2)


def test_offsets_behind_32_bits(rnn):
    """A pool of 2.1e9 elements: prefill and decode at its end, and moves from end to end.  Then a batch
    whose values, records and chunk states lie behind 2^31 elements or 2^32 bytes, training included."""
    Hk, Hv, K, V = 1, 8, 128, 128
    slots = 2 ** 31 // (Hv * V * K) + 3
    pool = torch.empty(slots, Hv, V, K, device="cuda")
    last = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    start = states(1, Hv, V, K, 1)
    pool[-1] = start[0]
    x = inputs(70, Hk, Hv, K, V, "bf16", 99)
    o, s = rnn.gated_delta_forward(*x.values(), s0=start, normalize=True)
    op, _ = rnn.gated_delta_forward(*x.values(), s0=pool, s_out=pool, slots=last, normalize=True)
    assert torch.equal(o, op) and torch.equal(s[0], pool[-1])
    one = [a[:, 0].contiguous() for a in x.values()]
    a, b = rnn.gated_delta_decode(*one, s, normalize=True), rnn.gated_delta_decode(*one, pool, slots=last,
                                                                                  normalize=True)
    assert torch.equal(a, b) and torch.equal(s[0], pool[-1])
    pool[0] = 1.0
    rnn.state_move(pool, torch.tensor([slots - 1, 0], dtype=torch.int32, device="cuda"),
                   torch.tensor([0, slots - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(s[0], pool[0]) and (pool[-1] == 1).all()
    del pool

    Hk, Hv, K, V = 1, 64, 64, 128
    T, short = 2 ** 31 // (Hv * V) + 64, 70
    total = T + short
    dt = torch.bfloat16
    g = torch.Generator("cuda").manual_seed(3)
    new = lambda *shape: torch.randn(shape, device="cuda", dtype=dt, generator=g)  # noqa: E731
    x = [new(1, total, Hk, K), new(1, total, Hk, K), new(1, total, Hv, V), -new(1, total, Hv).abs(),
         new(1, total, Hv).sigmoid()]
    cu = torch.tensor([0, T, total], dtype=torch.int32, device="cuda")
    d_o = new(1, total, Hv, V)
    o, s, ck, u = rnn.gated_delta_forward_train(*x, cu_seqlens=cu, normalize=True)
    grads = rnn.gated_delta_backward(*x, d_o, ck, u, cu_seqlens=cu, normalize=True)
    tail = [t[:, T:].contiguous() for t in x]
    to, ts, tck, tu = rnn.gated_delta_forward_train(*tail, normalize=True)
    want = rnn.gated_delta_backward(*tail, d_o[:, T:].contiguous(), tck, tu, normalize=True)
    close(o[:, T:], f64(to), "bf16", "o")
    close_state(s[1], f64(ts[0]), "bf16")
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, want):
        close(a[:, T:], f64(b), "bf16", name)
    close_state(grads[5][1], f64(want[5][0]), "bf16", "ds0")
    plain, _ = rnn.gated_delta_forward(*x, cu_seqlens=cu, normalize=True, want_state=False)
    assert torch.equal(plain[:, T - 200:], o[:, T - 200:])


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 64])
def test_decay_gradient_keeps_the_product_of_the_states(rnn, K, V, T):
    """With nothing written (beta = 0) and nothing read (d_o = 0), dg of every token is the whole decay
    times <S0, dS_T>: a sum of V K products of either sign, often small next to them.  The stored states
    keep 12 bits of significand for it, off by at most 2^-12: a product by 2^-11, and V K of them,
    uniformly and independently, by 2^-11 / sqrt(6) of their root sum of squares; six times that is 2^-9.7.
    (Factors of 8 bits would be off by 2^-8.3 in the mean.)"""
    B = 128
    x = inputs(B * T, 1, 1, K, V, "bf16", 111, B=B, slow=True)
    x["beta"].zero_()
    x["g"] *= 1 / T
    s0, ds = states(B, 1, V, K, 12), states(B, 1, V, K, 13)
    d_o = torch.zeros_like(x["v"])
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, normalize=True)
    dg = f64(rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, normalize=True)[3])[..., 0]
    c = np.exp(f64(x["g"])[..., 0].sum(1))
    terms = (f64(s0) * f64(ds)).reshape(B, -1)
    want, size = c * terms.sum(1), c * np.sqrt((terms ** 2).sum(1))
    off = np.abs(dg - want[:, None])
    assert (off <= 2.0 ** -8 * np.abs(want[:, None]) + 2.0 ** -9.7 * size[:, None]).all(), (off / size[:, None]).max()


def test_a_copy_of_the_stored_states_is_refused(rnn):
    x = inputs(100, 1, 1, 64, 64, "bf16", 112)
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values())
    d_o = torch.ones_like(o)
    rnn.gated_delta_backward(*x.values(), d_o, ck, u)
    for bad in (ck.contiguous(), ck.clone(), ck[:1], ck.float()):
        with pytest.raises(ValueError):
            rnn.gated_delta_backward(*x.values(), d_o, bad, u)


@pytest.mark.parametrize("layout", [("bf16", 64, 128, 1, 1), ("bf16", 128, 128, 1, 2), ("f32", 64, 64, 1, 1)], ids=str)
def test_gradients_of_a_sequence_in_segments(rnn, layout):
    """A training step whose forward is done in segments, next to a short and an empty sequence."""
    dtype, K, V, Hk, Hv = layout
    lens = [3300, 0, 70]
    cu = np.cumsum([0] + lens)
    x = inputs(int(cu[-1]), Hk, Hv, K, V, dtype, 120, slow=True)
    s0, ds = states(3, Hv, V, K, 1), states(3, Hv, V, K, 2)
    d_o = torch.from_numpy(np.random.default_rng(9).normal(size=(1, int(cu[-1]), Hv, V))).to(DT[dtype]).cuda()
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    need = rnn.gated_delta_forward_workspace_bytes
    assert need(int(cu[-1]), Hk, Hv, K, V, sequences=3, packed=True, dtype=dtype) > \
        need(64, 1, 1, K, V, dtype=dtype) * Hv * (int(cu[-1]) // 64 + 3)
    o, s, ck, u = rnn.gated_delta_forward_train(*x.values(), s0=s0, cu_seqlens=cut, normalize=True)
    grads = rnn.gated_delta_backward(*x.values(), d_o, ck, u, ds_T=ds, cu_seqlens=cut, normalize=True)
    for i in range(3):
        a, b = cu[i], cu[i + 1]
        want, S, trace = gd.forward(*rows(x, 0, a, b), f64(s0[i]), normalize=True)
        ref = gd.backward(*rows(x, 0, a, b), f64(d_o[0, a:b]), f64(ds[i]), f64(s0[i]), normalize=True)
        close(o[0, a:b], want, dtype, "o")
        close_state(s[i], S, dtype)
        for c in range((lens[i] + 63) // 64):
            close(ck[a // 64 + i + c], trace[64 * c], dtype, f"state {c} of sequence {i}")
        for name, got, w in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
            close(got[0, a:b], w, dtype, f"{name} of sequence {i}")
        close_state(grads[5][i], ref[5], dtype, "ds0")
