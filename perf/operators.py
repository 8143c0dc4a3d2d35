"""Operators measured on the GPU: the gated delta rule (prefill, single-token decode, training
step) and the moves of recurrent states between the slots of a pool.

Per sequence and value head, with a float32 state S [V, K], log decay g_t <= 0 and write
strength beta_t, each token computes

    Sd = exp(g_t) S;  e_t = v_t - Sd k_t;  S = Sd + beta_t e_t k_t^T;  o_t = scale S q_t

(value head h reads key head h // (Hv // Hk); with ``normalize`` q and k are divided by
sqrt(sum of squares + 1e-6) first).  ``run`` calls the framework's kernels where ``own`` is true
and computes the plain form in elementary float32 torch operations where it is false.
"""
import math

import torch

own = False

CHUNK = 64          # tokens per block of the plain form
NORM_EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # three short prompts of a small model arrive together: latency counts
        dict(name="prefill_short_ragged", op="prefill", dtype="bf16", seqs=3, longest=63, hk=2, hv=4,
             k=64, v=64, normalize=True, slots=True),
        # a serving step that continues 16 prompts of very different lengths in a state pool
        dict(name="prefill_serving_ragged", op="prefill", dtype="bf16", seqs=16, longest=2049, hk=16,
             hv=32, k=128, v=128, normalize=True, slots=True),
        # one long document, a layer of 32 value heads
        dict(name="prefill_long", op="prefill", dtype="bf16", seqs=1, longest=32768, hk=16, hv=32, k=128,
             v=128, normalize=True, slots=False),
        # batched prefill of the 2.9B width (40 heads of 64), keys normalised by the caller
        dict(name="prefill_batch_h40", op="prefill", dtype="bf16", seqs=8, longest=4096, hk=40, hv=40,
             k=64, v=64, normalize=False, slots=False),
        # float32 evaluation with rectangular states and an odd length
        dict(name="prefill_f32", op="prefill", dtype="f32", seqs=2, longest=1001, hk=4, hv=8, k=64, v=128,
             normalize=True, slots=False),
        # interactive decoding of a single sequence
        dict(name="decode_one", op="decode", dtype="bf16", seqs=1, hk=16, hv=32, k=128, v=128, normalize=True,
             slots=True),
        # a full serving batch of single tokens over a pool of resident states
        dict(name="decode_batch", op="decode", dtype="bf16", seqs=256, hk=16, hv=32, k=128, v=128,
             normalize=True, slots=True),
        # float32 decoding at an odd batch size
        dict(name="decode_f32", op="decode", dtype="f32", seqs=33, hk=12, hv=12, k=64, v=64, normalize=False,
             slots=False),
        # training step on one batch: forward, and every gradient
        dict(name="train_batch", op="train", dtype="bf16", seqs=4, longest=2048, hk=16, hv=32, k=128, v=128,
             normalize=True, ragged=False),
        # float32 training step on packed documents of odd lengths
        dict(name="train_f32_ragged", op="train", dtype="f32", seqs=3, longest=321, hk=2, hv=4, k=64, v=64,
             normalize=True, ragged=True),
        # beam search: the states of 16 beams of 4 follow their parents in every layer
        dict(name="move_beams", op="move", kind="beams", layers=12, pool=64, moves=64, heads=12, k=64, v=64),
        # a scheduler forks, compacts and frees slots of a 32-layer pool of the 2.9B width
        dict(name="move_scheduler", op="move", kind="mixed", layers=32, pool=96, moves=48, heads=40, k=64,
             v=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "decode", "train", "move"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    heads = dict(hk=_log_int(rng, 1, 16), k=rng.choice([64, 128]), v=rng.choice([64, 128]),
                 normalize=rng.random() < 0.5)
    heads["hv"] = heads["hk"] * rng.choice([1, 2, 4] if heads["hk"] <= 8 else [1, 2])
    if op == "decode":
        return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, 256), slots=rng.random() < 0.7, **heads)
    if op == "move":
        pool = _log_int(rng, 2, 200)
        return dict(op=op, kind=rng.choice(["beams", "mixed"]), layers=_log_int(rng, 1, 24), pool=pool,
                    moves=_log_int(rng, 1, pool), heads=_log_int(rng, 1, 16), k=rng.choice([64, 128]),
                    v=rng.choice([64, 128]))
    if op == "prefill":
        longest = _log_int(rng, 1, 16384 if dtype == "bf16" else 2048)
        most = 16384 if dtype == "bf16" else 4096
    else:
        longest = _log_int(rng, 1, 2048 if dtype == "bf16" else 512)
        most = 4096 if dtype == "bf16" else 1024
    case = dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, max(1, min(24, most // longest))), longest=longest,
                **heads)
    if op == "prefill":
        case["slots"] = rng.random() < 0.6
    else:
        case["ragged"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------------------------- inputs

def _lengths(case):
    """The sequences' lengths: ragged ones fall from the longest to about one, the same for every seed."""
    n, longest = case["seqs"], case["longest"]
    if not (case.get("slots") or case.get("ragged")):
        return [longest] * n
    return [max(1, int(longest * ((n - i) / n) ** 2)) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def order(n):
        return torch.rand(n, generator=gen, device="cuda").argsort().int()

    if case["op"] == "move":
        n, pool = case["moves"], case["pool"]
        state = normal(case["layers"], pool, case["heads"], case["v"], case["k"])
        if case["kind"] == "beams":
            # groups of four neighbouring slots: every beam continues one of its group's beams
            dst = torch.arange(n, device="cuda", dtype=torch.int32)
            pick = torch.randint(0, 4, (n,), generator=gen, device="cuda", dtype=torch.int32)
            src = torch.minimum(dst // 4 * 4 + pick, torch.full_like(dst, n - 1))
        else:
            # distinct targets; sources with repeats (forks), some of them targets too, and -1 (freed)
            dst = order(pool)[:n].contiguous()
            src = torch.randint(-1, pool, (n,), generator=gen, device="cuda", dtype=torch.int32)
            src = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.25, torch.full_like(src, -1), src)
        return dict(case=case, state=state, src=src, dst=dst)

    dt = TYPES[case["dtype"]]
    hk, hv, K, V = case["hk"], case["hv"], case["k"], case["v"]
    if case["op"] == "decode":
        lead = (case["seqs"],)
    else:
        lens = _lengths(case)
        packed = bool(case.get("slots") or case.get("ragged"))
        lead = (1, sum(lens)) if packed else (case["seqs"], case["longest"])
    q, k, v = normal(*lead, hk, K), normal(*lead, hk, K), normal(*lead, hv, V)
    if not case["normalize"]:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    # log decay -exp(A) softplus(x): heads forget over a few to some hundreds of tokens
    rate = torch.linspace(math.log(0.01), math.log(1.0), hv, device="cuda")
    g = -torch.exp(rate) * torch.nn.functional.softplus(normal(*lead, hv))
    beta = torch.sigmoid(normal(*lead, hv))
    state = dict(case=case, q=q.to(dt), k=k.to(dt), v=v.to(dt), g=g.to(dt), beta=beta.to(dt))
    if case["op"] == "decode":
        slots = case["seqs"] + case["seqs"] // 4 if case["slots"] else case["seqs"]
        state["pool"] = normal(slots, hv, V, K) * 0.3
        state["slots"] = order(slots)[:case["seqs"]].contiguous() if case["slots"] else None
        return state
    state["cu"] = None
    if packed:
        state["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    if case["op"] == "prefill":
        slots = case["seqs"] + 2 if case["slots"] else case["seqs"]
        state["pool"] = normal(slots, hv, V, K) * 0.3
        state["slots"] = order(slots)[:case["seqs"]].contiguous() if case["slots"] else None
    else:
        state["s0"] = normal(case["seqs"], hv, V, K) * 0.3
        state["do"] = normal(*lead, hv, V).to(dt)
        state["ds"] = normal(case["seqs"], hv, V, K) * 0.3
    return state


# ------------------------------------------------------------------------------- plain form

def _unit(x):
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) + NORM_EPS)


def _padded(x, cu, steps):
    """[sequences, heads, steps, ...] in float32 of a packed or dense [B, T, heads, ...], zeros behind each end."""
    if cu is None:
        x = x.float()
        short = steps - x.shape[1]
        if short:
            x = torch.cat([x, x.new_zeros(x.shape[0], short, *x.shape[2:])], 1)
        return x.transpose(1, 2)
    at = cu[:-1, None].long() + torch.arange(steps, device=cu.device)
    live = at < cu[1:, None]
    x = x[0][at.clamp(max=x.shape[1] - 1)].float()
    return torch.where(live.view(*live.shape, *[1] * (x.dim() - 2)), x, 0.0).transpose(1, 2)


def _packed(x, cu, total, dtype):
    """The reverse: [sequences, heads, steps, ...] back to the layout of the inputs."""
    x = x.transpose(1, 2)
    if cu is None:
        return x[:, :total].to(dtype).contiguous()
    at = cu[:-1, None].long() + torch.arange(x.shape[1], device=cu.device)
    return x[at < cu[1:, None]].to(dtype)[None]


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular blocks, by doubling the size of the inverted diagonal blocks."""
    n = A.shape[-1]
    i = torch.arange(n, device=A.device)
    X = torch.eye(n, device=A.device).expand_as(A)
    size = 1
    while size < n:
        low = (i[:, None] // (2 * size) == i[None] // (2 * size)) & (i[:, None] // size > i[None] // size)
        X = X - X @ torch.where(low, A, 0.0) @ X
        size *= 2
    return X


def _blocks(st):
    """Blocks of CHUNK tokens of the padded inputs, and what does not depend on the state."""
    case, cu = st["case"], st["cu"]
    steps = -(-case["longest"] // CHUNK) * CHUNK
    q, k, v, g, beta = (_padded(st[n], cu, steps) for n in ("q", "k", "v", "g", "beta"))
    rep = case["hv"] // case["hk"]
    qh, kh = (_unit(q), _unit(k)) if case["normalize"] else (q, k)
    n = steps // CHUNK

    def cut(x):
        return x.reshape(x.shape[0], x.shape[1], n, CHUNK, *x.shape[3:])

    Q, Kk = (cut(x.repeat_interleave(rep, 1)) for x in (qh, kh))
    V, g, beta = cut(v), cut(g), cut(beta)
    G = g.double().cumsum(-1)
    i = torch.arange(CHUNK, device=g.device)
    keep = i[:, None] >= i[None]
    E = torch.where(keep, torch.exp(torch.where(keep, G[..., :, None] - G[..., None, :], 0.0)), 0.0).float()
    grown = torch.exp(G).float()                      # decay from the block's start to each token
    rest = torch.exp(G[..., -1:] - G).float()         # decay from each token to the block's end
    KK = Kk @ Kk.transpose(-1, -2)
    A = torch.where(i[:, None] > i[None], beta[..., None] * E * KK, 0.0)
    scale = case["k"] ** -0.5
    P = scale * E * (Q @ Kk.transpose(-1, -2))
    return dict(n=n, q=q, k=k, Q=Q, K=Kk, V=V, beta=beta, E=E, KK=KK, grown=grown, rest=rest, A=A, T=_inverse(A),
                P=P, scale=scale, rep=rep)


def _plain_forward(b, S, keep=False):
    """The blocks one after the other (each needs the state that the last one left)."""
    outs, states, us = [], [], []
    for c in range(b["n"]):
        K, Q, beta, grown, rest = (b[x][:, :, c] for x in ("K", "Q", "beta", "grown", "rest"))
        St = S.transpose(-1, -2)
        R = beta[..., None] * (b["V"][:, :, c] - grown[..., None] * (K @ St))
        U = b["T"][:, :, c] @ R
        outs.append(b["scale"] * grown[..., None] * (Q @ St) + b["P"][:, :, c] @ U)
        if keep:
            states.append(S)
            us.append(U)
        S = grown[..., -1, None, None] * S + U.transpose(-1, -2) @ (rest[..., None] * K)
    return torch.cat(outs, 2), S, states, us


def _plain_prefill(st):
    b = _blocks(st)
    pool, slots = st["pool"], st["slots"]
    S = pool if slots is None else pool[slots.long()]
    O, S, _, _ = _plain_forward(b, S)
    o = _packed(O, st["cu"], st["case"]["longest"], st["q"].dtype)
    if slots is None:
        return o, S
    pool[slots.long()] = S
    return o, pool


def _plain_decode(st):
    case, pool, slots = st["case"], st["pool"], st["slots"]
    q, k, v, g, beta = (st[n].float() for n in ("q", "k", "v", "g", "beta"))
    if case["normalize"]:
        q, k = _unit(q), _unit(k)
    rep = case["hv"] // case["hk"]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    S = pool if slots is None else pool[slots.long()]
    S = torch.exp(g)[..., None, None] * S
    e = v - (S * k[..., None, :]).sum(-1)
    S = S + (beta[..., None] * e)[..., None] * k[..., None, :]
    o = case["k"] ** -0.5 * (S * q[..., None, :]).sum(-1)
    if slots is None:
        pool.copy_(S)
    else:
        pool[slots.long()] = S
    return o.to(st["q"].dtype), pool


def _plain_train(st):
    case, cu, dt = st["case"], st["cu"], st["q"].dtype
    b = _blocks(st)
    O, S_T, states, us = _plain_forward(b, st["s0"], keep=True)
    dO = _padded(st["do"], cu, b["n"] * CHUNK)
    dO = dO.reshape(*dO.shape[:2], b["n"], CHUNK, -1)
    D, scale = st["ds"], b["scale"]
    i = torch.arange(CHUNK, device=dO.device)
    strict = i[:, None] > i[None]
    got = []
    for c in reversed(range(b["n"])):
        K, Q, V, beta, grown, rest, E, P, T, A, KK = (
            b[x][:, :, c] for x in ("K", "Q", "V", "beta", "grown", "rest", "E", "P", "T", "A", "KK"))
        S, U, do = states[c], us[c], dO[:, :, c]
        gr, re, be = grown[..., None], rest[..., None], beta[..., None]
        KD = K @ D.transpose(-1, -2)
        dR = T.transpose(-1, -2) @ (P.transpose(-1, -2) @ do + re * KD)
        dP = do @ U.transpose(-1, -2)
        dA = torch.where(strict, -(dR @ U.transpose(-1, -2)), 0.0)
        doS, dRS = do @ S, dR @ S
        MP, MA = dP * (scale * E), dA * (be * E)
        dQ = scale * gr * doS + MP @ K
        UD = re * (U @ D)
        dK = -be * gr * dRS + UD + MP.transpose(-1, -2) @ Q + MA @ K + MA.transpose(-1, -2) @ K
        kS = (dRS * K).sum(-1) * grown
        dbeta = (dR * V).sum(-1) - kS + (dA * E * KK).sum(-1)
        # a decay at t lies on every path from a token before t (or the entry state) to one at or behind t
        M = dP * P + dA * A
        M = torch.where(strict, M, 0.0)
        pairs = torch.where(strict, M.flip(-2).cumsum(-2).flip(-2), 0.0).sum(-1)
        entry = scale * grown * (doS * Q).sum(-1) - beta * kS
        entry = entry.flip(-1).cumsum(-1).flip(-1)
        leave = (UD * K).sum(-1)
        leave = leave.cumsum(-1) - leave
        whole = (grown[..., -1] * (D * S).sum((-1, -2)))[..., None]
        got.append((dQ, dK, be * dR, pairs + entry + leave + whole, dbeta))
        D = gr[..., -1:, :] * D + scale * (do.transpose(-1, -2) @ (gr * Q)) \
            - dR.transpose(-1, -2) @ (be * gr * K)
    dq, dk, dv, dg, db = (torch.cat(x[::-1], 2) for x in zip(*got))

    def shared(d, x):
        """Heads that read the same key head add up; the norm's gradient where there is one."""
        d = d.reshape(d.shape[0], case["hk"], b["rep"], *d.shape[2:]).sum(2)
        if not case["normalize"]:
            return d
        unit, inv = _unit(x), torch.rsqrt(x.square().sum(-1, keepdim=True) + NORM_EPS)
        return inv * (d - unit * (unit * d).sum(-1, keepdim=True))

    total = case["longest"]
    return dict(o=_packed(O, cu, total, dt), s=S_T, dq=_packed(shared(dq, b["q"]), cu, total, dt),
                dk=_packed(shared(dk, b["k"]), cu, total, dt), dv=_packed(dv, cu, total, dt),
                dg=_packed(dg, cu, total, dt), dbeta=_packed(db, cu, total, dt), ds0=D)


def _plain_move(st):
    state, src, dst = st["state"], st["src"].long(), st["dst"].long()
    new = torch.where((src >= 0).view(1, -1, 1, 1, 1), state[:, src.clamp(min=0)], 0.0)
    state[:, dst] = new
    return state


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import linear_rnn_sequence_amd as rnn
        if op == "move":
            return rnn.state_move(st["state"], st["src"], st["dst"], slot_dim=1)
        x = (st["q"], st["k"], st["v"], st["g"], st["beta"])
        opts = dict(normalize=case["normalize"])
        if op == "decode":
            return rnn.gated_delta_decode(*x, st["pool"], slots=st["slots"], **opts), st["pool"]
        opts["cu_seqlens"] = st["cu"]
        if op == "prefill":
            into = st["pool"] if case["slots"] else None
            return rnn.gated_delta_forward(*x, s0=st["pool"], slots=st["slots"], s_out=into, **opts)
        o, s, ckpt, u = rnn.gated_delta_forward_train(*x, s0=st["s0"], **opts)
        dq, dk, dv, dg, dbeta, ds0 = rnn.gated_delta_backward(*x, st["do"], ckpt, u, ds_T=st["ds"], **opts)
        return dict(o=o, s=s, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, ds0=ds0)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "train": _plain_train, "move": _plain_move}[op](st)


# -------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "move":
        one = 4.0 * case["heads"] * case["k"] * case["v"] * case["layers"]
        return {"bytes": 2 * one * case["moves"], "flops": 0.0}
    size = 2 if case["dtype"] == "bf16" else 4
    hk, hv, K, V = case["hk"], case["hv"], case["k"], case["v"]
    tokens = case["seqs"] if case["op"] == "decode" else sum(_lengths(case))
    states = 4.0 * case["seqs"] * hv * V * K
    step = float(tokens) * hv * V * K
    ins = tokens * size * (2 * hk * K + hv * V + 2 * hv)
    out = tokens * size * hv * V
    if case["op"] == "train":
        # inputs and the output's gradient in, outputs and five gradients out; s0, its gradient, s, its gradient
        return {"bytes": 2 * ins + 2 * out + 4 * states, "flops": 20 * step}
    return {"bytes": ins + out + 2 * states, "flops": 6 * step}


# ------------------------------------------------------------------------------------- exact

def _per_token(x, cu, case):
    """Lists of float64 [sequences, value heads, ...] by step; a sequence that has ended gets zeros."""
    lens = _lengths(case)
    rows, at = [], 0
    for i, n in enumerate(lens):
        if cu is None:
            r = x[i].double()
        else:
            r = x[0, at:at + n].double()
            at += n
        rows.append(torch.nn.functional.pad(r, [0, 0] * (r.dim() - 1) + [0, case["longest"] - n]))
    x = torch.stack(rows, 1)
    return x if x.shape[2] == case["hv"] else x.repeat_interleave(case["hv"] // case["hk"], 2)


def _in_layout(x, cu, case):
    """The reverse of _per_token for a [steps, sequences, heads, ...] tensor."""
    if cu is None:
        return x.transpose(0, 1).contiguous()
    return torch.cat([x[:n, i] for i, n in enumerate(_lengths(case))])[None]


def _step(S, k, v, a, beta):
    Sd = a[..., None, None] * S
    e = v - torch.matmul(Sd, k[..., None])[..., 0]
    return Sd, e, torch.addcmul(Sd, (beta[..., None] * e)[..., None], k[..., None, :])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "move":
        new = st["state"].double()
        old = st["state"]
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            new[:, d] = old[:, s].double() if s >= 0 else 0.0
        return new
    scale = 1 / math.sqrt(case["k"])
    if case["op"] == "decode":
        x = [st[n].double() for n in ("q", "k", "v", "g", "beta")]
        x[:2] = [y.repeat_interleave(case["hv"] // case["hk"], 1) for y in x[:2]]
        if case["normalize"]:
            x[:2] = [y / (y.pow(2).sum(-1, keepdim=True) + NORM_EPS).sqrt() for y in x[:2]]
        pool = st["pool"].double()
        at = torch.arange(case["seqs"], device="cuda") if st["slots"] is None else st["slots"].long()
        S = _step(pool[at], x[1], x[2], x[3].exp(), x[4])[2]
        pool[at] = S
        return scale * torch.matmul(S, x[0][..., None])[..., 0], pool
    cu, T = st["cu"], case["longest"]
    q, k, v, g, beta = (_per_token(st[n], cu, case) for n in ("q", "k", "v", "g", "beta"))
    raw = {"q": q, "k": k}
    if case["normalize"]:
        q, k = (y / (y.pow(2).sum(-1, keepdim=True) + NORM_EPS).sqrt() for y in (q, k))
    a = g.exp()
    if case["op"] == "prefill":
        at = torch.arange(case["seqs"], device="cuda") if st["slots"] is None else st["slots"].long()
        S = st["pool"].double()[at]
    else:
        S = st["s0"].double()
    os, kept, every = [], [], 32
    for t in range(T):
        if t % every == 0:
            kept.append(S)
        S = _step(S, k[t], v[t], a[t], beta[t])[2]
        os.append(scale * torch.matmul(S, q[t][..., None])[..., 0])
        if case["op"] == "prefill":
            kept.clear()
    o = _in_layout(torch.stack(os), cu, case)
    if case["op"] == "prefill":
        if st["slots"] is None:
            return o, S
        pool = st["pool"].double()
        pool[at] = S
        return o, pool
    do = _per_token(st["do"], cu, case)
    D, S_T = st["ds"].double(), S
    grads = {n: [None] * T for n in ("dq", "dk", "dv", "dg", "dbeta")}
    for first in reversed(range(0, T, every)):
        S, held = kept[first // every], []
        for t in range(first, min(T, first + every)):
            held.append(S)
            S = _step(S, k[t], v[t], a[t], beta[t])[2]
        for t in reversed(range(first, min(T, first + every))):
            prev = held[t - first]
            Sd, e, S = _step(prev, k[t], v[t], a[t], beta[t])
            D = torch.addcmul(D, scale * do[t][..., None], q[t][..., None, :])
            grads["dq"][t] = scale * torch.matmul(S.transpose(-1, -2), do[t][..., None])[..., 0]
            Dk = torch.matmul(D, k[t][..., None])[..., 0]
            grads["dbeta"][t] = (e * Dk).sum(-1)
            de = beta[t][..., None] * Dk
            grads["dv"][t] = de
            grads["dk"][t] = torch.matmul(D.transpose(-1, -2), (beta[t][..., None] * e)[..., None])[..., 0] \
                - torch.matmul(Sd.transpose(-1, -2), de[..., None])[..., 0]
            D = torch.addcmul(D, de[..., None], k[t][..., None, :], value=-1)
            grads["dg"][t] = (D * Sd).sum((-1, -2))
            D = a[t][..., None, None] * D
    out = {"o": o, "s": S_T, "ds0": D}
    for n, rows in grads.items():
        d = torch.stack(rows)
        if n in ("dq", "dk"):
            x = raw[n[1]]
            if case["normalize"]:
                r = (x.pow(2).sum(-1, keepdim=True) + NORM_EPS).sqrt()
                d = d / r - x * (x * d).sum(-1, keepdim=True) / r.pow(3)
            d = d.unflatten(2, (case["hk"], -1)).sum(3)
        out[n] = _in_layout(d, cu, case)
    return out
