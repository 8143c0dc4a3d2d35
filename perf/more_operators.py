"""Operators measured on the GPU: linear attention with a decay for each head (prefill,
single-token decode, training step) and the group norm with an activation behind it.

Linear attention: per sequence and value head h, with a float32 state S [V, K] and the head's log
decay g_h <= 0, each token computes

    S = exp(g_h) S + v_t k_t^T;  o_t = scale S q_t

(value head h reads key head h // (Hv // Hk); scale = K^-0.5).  Group norm: each row x [C] by
itself, in groups of channels (a head's), n = (x - mean) / sqrt(var + eps) weight + bias
(``rms``: x / sqrt(mean(x^2) + eps)), y = n act(gate) with a gate, act(n) without one.  ``run``
calls the framework's kernels where ``own`` is true and computes the plain form in elementary
float32 torch operations where it is false.
"""
import math

import torch

own = False

CHUNK = 64          # tokens per block of the plain form
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # three short prompts of a small model arrive together: latency counts
        dict(name="prefill_short_ragged", op="prefill", dtype="bf16", seqs=3, longest=63, hk=2, hv=4,
             k=64, v=64, slots=True),
        # a serving step that continues 16 prompts of very different lengths in a state pool
        dict(name="prefill_serving_ragged", op="prefill", dtype="bf16", seqs=16, longest=2049, hk=32,
             hv=32, k=128, v=128, slots=True),
        # one long document, a layer of 32 heads
        dict(name="prefill_long", op="prefill", dtype="bf16", seqs=1, longest=32768, hk=32, hv=32, k=128,
             v=128, slots=False),
        # batched prefill of the 2.9B width (40 heads of 64)
        dict(name="prefill_batch_h40", op="prefill", dtype="bf16", seqs=8, longest=4096, hk=40, hv=40,
             k=64, v=64, slots=False),
        # float32 evaluation with rectangular states, shared key heads and an odd length
        dict(name="prefill_f32", op="prefill", dtype="f32", seqs=2, longest=1001, hk=4, hv=8, k=64, v=128,
             slots=False),
        # interactive decoding of a single sequence
        dict(name="decode_one", op="decode", dtype="bf16", seqs=1, hk=32, hv=32, k=128, v=128, slots=True),
        # a full serving batch of single tokens over a pool of resident states
        dict(name="decode_batch", op="decode", dtype="bf16", seqs=256, hk=32, hv=32, k=128, v=128,
             slots=True),
        # training step on one batch: forward, and every gradient
        dict(name="train_batch", op="train", dtype="bf16", seqs=4, longest=2048, hk=32, hv=32, k=128, v=128,
             ragged=False),
        # float32 training step on packed documents of odd lengths, shared key heads
        dict(name="train_f32_ragged", op="train", dtype="f32", seqs=3, longest=321, hk=2, hv=4, k=64, v=64,
             ragged=True),
        # the norm and gate behind a decoding step of seven sequences
        dict(name="norm_decode", op="norm", dtype="bf16", rows=7, groups=32, size=128, gate=True,
             act="silu", rms=False, affine=True),
        # the same behind the prefill of a large batch
        dict(name="norm_prefill", op="norm", dtype="bf16", rows=32768, groups=32, size=128, gate=True,
             act="silu", rms=False, affine=True),
        # training step at the 2.9B width: the norm with its gate, and every gradient
        dict(name="norm_train_h40", op="norm_train", dtype="bf16", rows=8191, groups=40, size=64, gate=True,
             act="silu", rms=False, affine=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "train", "train", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_train"):
        return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 4096), groups=_log_int(rng, 1, 40),
                    size=rng.choice([32, 50, 64, 80, 99, 128, 128, 200, 256]), gate=rng.random() < 0.7,
                    act=rng.choice(["silu", "silu", "sigmoid", "none"]), rms=rng.random() < 0.3,
                    affine=rng.random() < 0.8)
    heads = dict(hk=_log_int(rng, 1, 16), k=rng.choice([64, 128]), v=rng.choice([64, 128, 128, 192, 256]))
    heads["hv"] = heads["hk"] * rng.choice([1, 1, 2, 4] if heads["hk"] <= 8 else [1, 1, 2])
    if op == "decode":
        return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, 128), slots=rng.random() < 0.7, **heads)
    if op == "prefill":
        longest = _log_int(rng, 1, 16384 if dtype == "bf16" else 2048)
        most = 16384 if dtype == "bf16" else 4096
    else:
        longest = _log_int(rng, 1, 2048 if dtype == "bf16" else 512)
        most = 4096 if dtype == "bf16" else 1024
    case = dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, max(1, min(24, most // longest))), longest=longest,
                **heads)
    case["slots" if op == "prefill" else "ragged"] = rng.random() < 0.6
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
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def order(n):
        return torch.rand(n, generator=gen, device="cuda").argsort().int()

    if case["op"] in ("norm", "norm_train"):
        rows, C = case["rows"], case["groups"] * case["size"]
        # readouts of a recurrence: every head has a size and an offset of its own
        x = normal(rows, C) * torch.exp(normal(case["groups"])).repeat_interleave(case["size"]) + 0.2 * normal(C)
        state = dict(case=case, x=x.to(dt), gate=normal(rows, C).to(dt) if case["gate"] else None,
                     weight=1 + 0.1 * normal(C) if case["affine"] else None,
                     bias=0.1 * normal(C) if case["affine"] else None)
        if case["op"] == "norm_train":
            state["dy"] = normal(rows, C).to(dt)
        return state

    hk, hv, K, V = case["hk"], case["hv"], case["k"], case["v"]
    if case["op"] == "decode":
        lead = (case["seqs"],)
    else:
        lens = _lengths(case)
        packed = bool(case.get("slots") or case.get("ragged"))
        lead = (1, sum(lens)) if packed else (case["seqs"], case["longest"])
    # heads that forget over two to some thousands of tokens, a little different from layer to layer
    g = -torch.exp2(-1 - torch.arange(hv, device="cuda") * (10 / hv) - torch.rand(hv, generator=gen, device="cuda"))
    state = dict(case=case, q=normal(*lead, hk, K).to(dt), k=normal(*lead, hk, K).to(dt),
                 v=normal(*lead, hv, V).to(dt), g=g)
    if case["op"] == "decode":
        slots = case["seqs"] + case["seqs"] // 4 if case["slots"] else case["seqs"]
        state["pool"] = normal(slots, hv, V, K)
        state["slots"] = order(slots)[:case["seqs"]].contiguous() if case["slots"] else None
        return state
    state["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).int() if packed else None
    if case["op"] == "prefill":
        slots = case["seqs"] + 2 if case["slots"] else case["seqs"]
        state["pool"] = normal(slots, hv, V, K)
        state["slots"] = order(slots)[:case["seqs"]].contiguous() if case["slots"] else None
    else:
        state["s0"] = normal(case["seqs"], hv, V, K)
        state["do"] = normal(*lead, hv, V).to(dt)
        state["ds"] = normal(case["seqs"], hv, V, K)
    return state


# ------------------------------------------------------------------------------- plain form

def _padded(x, cu, steps):
    """[sequences, heads, blocks, CHUNK, channels] in float32 of a packed or dense [B, T, heads, channels],
    zeros behind each end."""
    if cu is None:
        x = x.float()
        short = steps - x.shape[1]
        if short:
            x = torch.cat([x, x.new_zeros(x.shape[0], short, *x.shape[2:])], 1)
    else:
        at = cu[:-1, None].long() + torch.arange(steps, device=cu.device)
        live = at < cu[1:, None]
        x = torch.where(live[..., None, None], x[0][at.clamp(max=x.shape[1] - 1)].float(), 0.0)
    return x.unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, 4)


def _packed(x, cu, total, dtype):
    """The reverse: back to the layout of the inputs."""
    x = x.permute(0, 2, 3, 1, 4).flatten(1, 2)
    if cu is None:
        return x[:, :total].to(dtype).contiguous()
    at = cu[:-1, None].long() + torch.arange(x.shape[1], device=cu.device)
    return x[at < cu[1:, None]].to(dtype)[None]


def _blocks(st):
    """Blocks of CHUNK tokens, and the decays between their tokens.  A token's number counts up to its
    sequence's end, so that the zeros behind it change nothing."""
    case, cu = st["case"], st["cu"]
    steps = -(-case["longest"] // CHUNK) * CHUNK
    q, k, v = (_padded(st[n], cu, steps) for n in ("q", "k", "v"))
    rep = case["hv"] // case["hk"]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    device = q.device
    if cu is None:
        length = torch.full((q.shape[0], 1), case["longest"], device=device)
    else:
        length = (cu[1:] - cu[:-1])[:, None].long()
    count = torch.minimum(torch.arange(1, steps + 1, device=device)[None], length).unflatten(1, (-1, CHUNK))
    bound = torch.minimum(torch.arange(0, steps + 1, CHUNK, device=device)[None], length)   # [sequences, n + 1]
    i, b = torch.arange(CHUNK, device=device), torch.arange(bound.shape[1], device=device)
    g = st["g"].double()

    def power(x, keep=None):
        """(x, decay^x) per head, zero where not kept; x [sequences, ...]."""
        x = x[:, None].double()
        d = torch.exp(g.view(-1, *[1] * (x.dim() - 2)) * x)
        return x.float(), (d if keep is None else torch.where(keep, d, 0.0)).float()

    return dict(
        q=q, k=k, v=v, scale=case["k"] ** -0.5, rep=rep,
        pair=power((count[..., :, None] - count[..., None, :]).clamp(min=0), i[:, None] >= i[None]),
        enter=power(count - bound[:, :-1, None]),         # from the block's start to each token
        leave=power(bound[:, 1:, None] - count),          # from each token to the block's end
        first=power(bound),                               # from the sequence's start to each bound
        last=power(length - bound),                       # from each bound to the sequence's end
        # from block c's end to bound b, and from bound b to block c's start
        since=power((bound[:, :, None] - bound[:, None, 1:]).clamp(min=0), b[:, None] > b[None, :-1]),
        until=power((bound[:, None, :-1] - bound[:, :, None]).clamp(min=0), b[:, None] <= b[None, :-1]))


def _apply(matrix, x):
    """[..., n + 1, n] times the blocks' states [..., n, V, K]."""
    return (matrix @ x.flatten(-2)).unflatten(-1, x.shape[-2:])


def _write(b, factor):
    """What each block adds to the state, its tokens weighted."""
    return b["v"].transpose(-1, -2) @ (factor[..., None] * b["k"])


def _forward(b, s0):
    """Readouts, and the states at all bounds."""
    S = _apply(b["since"][1], _write(b, b["leave"][1])) + b["first"][1][..., None, None] * s0[:, :, None]
    P = b["scale"] * b["pair"][1] * (b["q"] @ b["k"].transpose(-1, -2))
    inter = b["q"] @ S[:, :, :-1].transpose(-1, -2)
    return b["scale"] * b["enter"][1][..., None] * inter + P @ b["v"], S, P, inter


def _plain_prefill(st):
    b = _blocks(st)
    pool, slots = st["pool"], st["slots"]
    o, S, _, _ = _forward(b, pool if slots is None else pool[slots.long()])
    o = _packed(o, st["cu"], st["case"]["longest"], st["q"].dtype)
    if slots is None:
        return o, S[:, :, -1].contiguous()
    pool[slots.long()] = S[:, :, -1]
    return o, pool


def _plain_decode(st):
    case, pool, slots = st["case"], st["pool"], st["slots"]
    rep = case["hv"] // case["hk"]
    q, k = (st[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    S = pool if slots is None else pool[slots.long()]
    S = torch.exp(st["g"])[:, None, None] * S + st["v"].float()[..., None] * k[..., None, :]
    o = case["k"] ** -0.5 * (S * q[..., None, :]).sum(-1)
    if slots is None:
        pool.copy_(S)
    else:
        pool[slots.long()] = S
    return o.to(st["q"].dtype), pool


def _plain_train(st):
    case, cu, dt = st["case"], st["cu"], st["q"].dtype
    b = _blocks(st)
    q, k, v, scale = b["q"], b["k"], b["v"], b["scale"]
    o, S, P, inter = _forward(b, st["s0"])
    do = _padded(st["do"], cu, q.shape[2] * CHUNK)
    far, enter = b["enter"]
    reads = scale * (do.transpose(-1, -2) @ (enter[..., None] * q))
    D = _apply(b["until"][1], reads) + b["last"][1][..., None, None] * st["ds"][:, :, None]
    dA = scale * b["pair"][1] * (do @ v.transpose(-1, -2))
    exit, leave = D[:, :, 1:], b["leave"][1]
    dq = scale * enter[..., None] * (do @ S[:, :, :-1]) + dA @ k
    dk = leave[..., None] * (v @ exit) + dA.transpose(-1, -2) @ q
    dv = leave[..., None] * (k @ exit.transpose(-1, -2)) + P.transpose(-1, -2) @ do
    # the states' derivatives by g: every decay^x becomes x decay^x
    x, d = b["since"]
    R = _apply(x * d, _write(b, leave)) + _apply(d, _write(b, b["leave"][0] * leave))
    R = R + (b["first"][0] * b["first"][1])[..., None, None] * st["s0"][:, :, None]
    moved = far[..., None] * inter + q @ R[:, :, :-1].transpose(-1, -2)
    dg = (b["pair"][0] * dA * (q @ k.transpose(-1, -2))).double().sum((0, 2, 3, 4)) \
        + (scale * enter[..., None] * moved * do).double().sum((0, 2, 3, 4)) \
        + (R[:, :, -1] * st["ds"]).double().sum((0, 2, 3))

    def shared(d):
        return d.unflatten(1, (case["hk"], b["rep"])).sum(2)

    total = case["longest"]
    return dict(o=_packed(o, cu, total, dt), s=S[:, :, -1].contiguous(), dq=_packed(shared(dq), cu, total, dt),
                dk=_packed(shared(dk), cu, total, dt), dv=_packed(dv, cu, total, dt), dg=dg.float(),
                ds0=D[:, :, 0].contiguous())


def _act(x, name):
    """The activation and its derivative."""
    if name == "none":
        return x, torch.ones_like(x)
    s = torch.sigmoid(x)
    return (s, s * (1 - s)) if name == "sigmoid" else (x * s, s * (1 + x * (1 - s)))


def _plain_norm(st):
    case, dt = st["case"], st["x"].dtype
    shape = (case["rows"], case["groups"], case["size"])
    x = st["x"].float().view(shape)
    if not case["rms"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    unit = (x * rstd).view(st["x"].shape)
    n = unit if st["weight"] is None else unit * st["weight"] + st["bias"]
    a, da = _act(n if st["gate"] is None else st["gate"].float(), case["act"])
    y = a if st["gate"] is None else n * a
    if case["op"] == "norm":
        return y.to(dt)
    dy = st["dy"].float()
    dn = dy * (da if st["gate"] is None else a)
    du = dn if st["weight"] is None else dn * st["weight"]
    u, d = unit.view(shape), du.view(shape)
    dx = d - u * (u * d).mean(-1, keepdim=True)
    if not case["rms"]:
        dx = dx - d.mean(-1, keepdim=True)
    out = dict(y=y.to(dt), dx=(rstd * dx).view(st["x"].shape).to(dt))
    if st["weight"] is not None:
        out.update(dweight=(dn * unit).sum(0), dbias=dn.sum(0))
    if st["gate"] is not None:
        out["dgate"] = (dy * n * da).to(dt)
    return out


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import linear_rnn_sequence_amd as rnn
        if op in ("norm", "norm_train"):
            affine = dict(weight=st["weight"], bias=st["bias"], gate=st["gate"], activation=case["act"],
                          rms=case["rms"], eps=EPS)
            y = rnn.group_norm_forward(st["x"], case["groups"], **affine)
            if op == "norm":
                return y
            dx, dweight, dbias, dgate = rnn.group_norm_backward(st["x"], case["groups"], st["dy"], **affine)
            out = dict(y=y, dx=dx, dweight=dweight, dbias=dbias, dgate=dgate)
            return {n: t for n, t in out.items() if t is not None}
        x = (st["q"], st["k"], st["v"], st["g"])
        if op == "decode":
            return rnn.linear_attention_decode(*x, st["pool"], slots=st["slots"]), st["pool"]
        if op == "prefill":
            into = st["pool"] if case["slots"] else None
            return rnn.linear_attention_forward(*x, s0=st["pool"], slots=st["slots"], s_out=into,
                                                cu_seqlens=st["cu"])
        o, s = rnn.linear_attention_forward(*x, s0=st["s0"], cu_seqlens=st["cu"])
        dq, dk, dv, dg, ds0 = rnn.linear_attention_backward(*x, st["do"], s0=st["s0"], ds_T=st["ds"],
                                                            cu_seqlens=st["cu"])
        return dict(o=o, s=s, dq=dq, dk=dk, dv=dv, dg=dg, ds0=ds0)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "train": _plain_train, "norm": _plain_norm,
            "norm_train": _plain_norm}[op](st)


# -------------------------------------------------------------------------------------- work

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        n = float(case["rows"] * case["groups"] * case["size"])
        params = 8.0 * case["groups"] * case["size"] * case["affine"]
        tensors = 2 + case["gate"]
        if case["op"] == "norm":
            return {"bytes": tensors * size * n + params, "flops": 15 * n}
        # x, gate, dy in, y, dx, dgate out
        return {"bytes": (tensors + 2 + case["gate"]) * size * n + 2 * params, "flops": 45 * n}
    hk, hv, K, V = case["hk"], case["hv"], case["k"], case["v"]
    tokens = case["seqs"] if case["op"] == "decode" else sum(_lengths(case))
    states = 4.0 * case["seqs"] * hv * V * K
    step = float(tokens) * hv * V * K
    ins, out = tokens * size * (2.0 * hk * K + hv * V), tokens * size * hv * float(V)
    if case["op"] == "train":
        # inputs and the output's gradient in, outputs and gradients out; s0, its gradient, s, its gradient
        return {"bytes": 2 * ins + 2 * out + 4 * states, "flops": 15 * step}
    return {"bytes": ins + out + 2 * states, "flops": 5 * step}


# ------------------------------------------------------------------------------------- exact

def _per_token(x, case):
    """[steps, sequences, value heads, channels] in float64; a sequence that has ended gets zeros."""
    lens = _lengths(case)
    if x.shape[0] == 1:
        rows = torch.split(x[0], lens)
    else:
        rows = list(x)
    x = torch.stack([torch.nn.functional.pad(r.double(), (0, 0, 0, 0, 0, case["longest"] - len(r)))
                     for r in rows], 1)
    return x if x.shape[2] == case["hv"] else x.repeat_interleave(case["hv"] // case["hk"], 2)


def _in_layout(rows, case, packed, heads):
    """The reverse, for a list of the steps; heads that read the same key head add up."""
    x = torch.stack(rows)
    x = x.unflatten(2, (heads, -1)).sum(3)
    if packed:
        return torch.cat([x[:n, i] for i, n in enumerate(_lengths(case))])[None]
    return x.transpose(0, 1).contiguous()


def _exact_norm(st):
    case, x = st["case"], st["x"].double()
    C = x.shape[1]
    groups = x.reshape(-1, case["size"])
    mean = torch.zeros_like(groups[:, :1]) if case["rms"] else groups.sum(1, keepdim=True) / case["size"]
    var = ((groups - mean) ** 2).sum(1, keepdim=True) / case["size"]
    inv = 1 / (var + EPS).sqrt()
    unit = (groups - mean) * inv
    weight = torch.ones(C, device="cuda").double() if st["weight"] is None else st["weight"].double()
    bias = torch.zeros_like(weight) if st["bias"] is None else st["bias"].double()
    n = unit.reshape(-1, C) * weight + bias
    z = n if st["gate"] is None else st["gate"].double()
    sig = 1 / (1 + torch.exp(-z))
    act, slope = {"none": (z, z * 0 + 1), "sigmoid": (sig, sig - sig * sig),
                  "silu": (z * sig, sig + z * (sig - sig * sig))}[case["act"]]
    y = act if st["gate"] is None else n * act
    if case["op"] == "norm":
        return y
    dy = st["dy"].double()
    dn = dy * slope if st["gate"] is None else dy * act
    du = (dn * weight).reshape(-1, case["size"])
    along = (du * unit).sum(1, keepdim=True) / case["size"]
    dx = du - unit * along
    if not case["rms"]:
        dx = dx - du.sum(1, keepdim=True) / case["size"]
    out = dict(y=y, dx=(dx * inv).reshape(-1, C))
    if st["weight"] is not None:
        out["dweight"] = (dn * unit.reshape(-1, C)).sum(0)
        out["dbias"] = dn.sum(0)
    if st["gate"] is not None:
        out["dgate"] = dy * n * slope
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(st)
    scale = 1 / math.sqrt(case["k"])
    decay = torch.exp(st["g"].double())[None, :, None, None]
    if case["op"] == "decode":
        rep = case["hv"] // case["hk"]
        q, k = (st[n].double().repeat_interleave(rep, 1) for n in ("q", "k"))
        pool = st["pool"].double()
        at = torch.arange(case["seqs"], device="cuda") if st["slots"] is None else st["slots"].long()
        S = pool[at] * decay + st["v"].double()[..., None] * k[..., None, :]
        pool[at] = S
        return scale * torch.matmul(S, q[..., None])[..., 0], pool
    T, packed, train = case["longest"], st["cu"] is not None, case["op"] == "train"
    q, k, v = (_per_token(st[n], case) for n in ("q", "k", "v"))
    lens = torch.tensor(_lengths(case), device="cuda")[:, None, None, None]
    if train:
        S, do, dg, R = st["s0"].double(), _per_token(st["do"], case), 0.0, 0.0
    else:
        at = torch.arange(case["seqs"], device="cuda") if st["slots"] is None else st["slots"].long()
        S = st["pool"].double()[at]
    even = len(set(_lengths(case))) == 1
    os, dqs = [], []
    for t in range(T):
        a = decay if even else torch.where(t < lens, decay, 1.0)     # a sequence that has ended keeps its state
        if train:
            R = decay * (R + S) if even else torch.where(t < lens, decay * (R + S), R)
        S = torch.addcmul(a * S, v[t][..., None], k[t][..., None, :])
        os.append(scale * torch.matmul(S, q[t][..., None])[..., 0])
        if train:
            dqs.append(scale * torch.matmul(S.transpose(-1, -2), do[t][..., None])[..., 0])
            dg = dg + scale * (torch.matmul(R, q[t][..., None])[..., 0] * do[t]).sum((0, 2))
    o = _in_layout(os, case, packed, case["hv"])
    if not train:
        if st["slots"] is None:
            return o, S
        pool = st["pool"].double()
        pool[at] = S
        return o, pool
    D = st["ds"].double()
    dg = dg + (R * D).sum((0, 2, 3))
    dks, dvs = [None] * T, [None] * T
    for t in reversed(range(T)):
        D = torch.addcmul(D, scale * do[t][..., None], q[t][..., None, :])
        dks[t] = torch.matmul(D.transpose(-1, -2), v[t][..., None])[..., 0]
        dvs[t] = torch.matmul(D, k[t][..., None])[..., 0]
        D = D * (decay if even else torch.where(t < lens, decay, 1.0))
    hk, hv = case["hk"], case["hv"]
    return dict(o=o, s=S, dq=_in_layout(dqs, case, packed, hk), dk=_in_layout(dks, case, packed, hk),
                dv=_in_layout(dvs, case, packed, hv), dg=dg, ds0=D)
