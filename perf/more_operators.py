"""The operators of a linear attention layer around its projections, as cases to
time and to compare: linear attention with a constant decay for each head
(``linear_attn_*``) and the norm over groups of channels with its gate
(``group_norm_*``), each for prompts, for training and for single tokens.

``run`` computes them either as plain 32-bit torch arithmetic (``own`` false)
or through this repository's entry points (``own`` true); ``exact`` gives the
same values from the definitions in 64 bits.

Queries are [batch, seqlen, heads, key], keys and values [batch, seqlen,
kv_heads, key or value], states [batch, heads, value, key].  Head h reads the
key and value head h * kv_heads // heads; len_b is the length of sequence b.

    attention   S[t] = e^log_decay S[t-1] + v[t] k[t]^T,  y[t] = scale S[t] q[t]
    norm        over each group's channels of one row, with act = silu or identity:
                n = (x - mean) / sqrt(var + eps)  (mean 0 unless centred), p = weight n + bias
                y = act(p), or p act(gate), or p with x act(gate) in the place of x

Steps t >= len_b are no part of the sequence: outputs and gradients are zero
there, and the final state is the one after step len_b - 1.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-5


def listed():
    return [
        # a short prompt of one user, 12 heads of 128: latency
        dict(name="attn_fwd prompt 96", op="attn_fwd", batch=1, seqlen=96, heads=12, kv_heads=12, key=128, value=128,
             dtype=BF16, ragged=False, carry=False),
        # training forward at width 5120, 40 heads of 128
        dict(name="attn_fwd 8x2048", op="attn_fwd", batch=8, seqlen=2048, heads=40, kv_heads=40, key=128, value=128,
             dtype=BF16, ragged=False, carry=False),
        # one long document continued from a state, few heads: one sequence has to fill the card
        dict(name="attn_fwd 1x32768", op="attn_fwd", batch=1, seqlen=32768, heads=12, kv_heads=12, key=128, value=128,
             dtype=BF16, ragged=False, carry=True),
        # fp32, odd sizes, unequal sequences, three heads to a key and value head
        dict(name="attn_fwd odd f32", op="attn_fwd", batch=3, seqlen=517, heads=6, kv_heads=2, key=40, value=75,
             dtype=F32, ragged=True, carry=True),
        # a training step's backward at width 5120
        dict(name="attn_bwd 4x2048", op="attn_bwd", batch=4, seqlen=2048, heads=40, kv_heads=40, key=128, value=128,
             dtype=BF16, ragged=False, carry=False),
        # gradients of unequal sequences with shared key and value heads of 64, states carried in and out
        dict(name="attn_bwd ragged shared", op="attn_bwd", batch=3, seqlen=1301, heads=16, kv_heads=4, key=64, value=64,
             dtype=BF16, ragged=True, carry=True),
        # one token of one request: latency
        dict(name="attn_step 1", op="attn_step", batch=1, heads=12, kv_heads=12, key=128, value=128, dtype=BF16),
        # one token of 256 requests
        dict(name="attn_step 256", op="attn_step", batch=256, heads=40, kv_heads=40, key=128, value=128, dtype=BF16),
        # one token of one request through the gated norm of 40 heads: latency
        dict(name="norm_fwd 1", op="norm_fwd", batch=1, seqlen=1, channels=5120, groups=40, dtype=BF16, ragged=False,
             form="gate", center=True, affine=True),
        # the gated norm after the attention, a group to a head
        dict(name="norm_fwd 8x4096", op="norm_fwd", batch=8, seqlen=4096, channels=5120, groups=40, dtype=BF16,
             ragged=False, form="gate", center=True, affine=True),
        # the norm of the state space layer: the gate first, no mean, the whole row
        dict(name="norm_bwd 4x2048", op="norm_bwd", batch=4, seqlen=2048, channels=5120, groups=1, dtype=BF16,
             ragged=False, form="gate_first", center=False, affine=True),
        # fp32, odd sizes, unequal sequences, the activation on the norm itself
        dict(name="norm_bwd odd f32", op="norm_bwd", batch=3, seqlen=517, channels=771, groups=3, dtype=F32,
             ragged=True, form="plain", center=True, affine=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    half = 1 if dtype == BF16 else 2
    if op.startswith("norm"):
        groups = rng.choice([1, 1, 2, 3, 8, 40])
        channels = groups * spread(max(1, 64 // groups), 5120 // groups)
        if rng.random() < 0.6:
            channels += -channels % (64 * groups) if groups < 40 else -channels % (8 * groups)
        case = dict(op=op, batch=spread(1, 8), seqlen=spread(1, 4096), channels=channels, groups=groups, dtype=dtype,
                    ragged=rng.random() < 0.4, form=rng.choice(["gate", "gate_first", "plain"]),
                    center=rng.random() < 0.5, affine=rng.random() < 0.8)
        most = (8 * 4096 if op == "norm_fwd" else 4 * 2048) * 5120 // half
        while case["batch"] * case["seqlen"] * channels > most:
            case["seqlen"] = case["seqlen"] // 2 + 1
        return case
    kv_heads = spread(1, 40)
    heads = kv_heads * (rng.choice([2, 3, 4]) if kv_heads <= 10 and rng.random() < 0.4 else 1)
    key, value = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (256, 256),
                             (rng.randint(1, 256), rng.randint(1, 256))])
    case = dict(op=op, batch=spread(1, 256 if op == "attn_step" else 8), heads=heads, kv_heads=kv_heads, key=key,
                value=value, dtype=dtype)
    if op == "attn_step":
        while case["batch"] * heads * key * value > 256 * 40 * 128 * 128:
            case["batch"] = case["batch"] // 2 + 1
        return case
    case.update(seqlen=spread(1, 32768), ragged=rng.random() < 0.4, carry=rng.random() < 0.5)
    # at most the rows, the elements and the operations of the largest listed case
    rows = (8 if op == "attn_fwd" else 4) * 2048 * 40 // half

    def over():
        n = case["batch"] * case["seqlen"] * heads
        return max(n, n * (key + value) // 256, n * key * value // 128 ** 2) > rows
    while over():
        if case["seqlen"] > 64 or case["batch"] == 1:
            case["seqlen"] = case["seqlen"] // 2 + 1
        else:
            case["batch"] -= 1
    return case


# ---- sizes and inputs ------------------------------------------------------------

def _lengths(case, gen):
    """Unequal lengths, one of them the whole and, where there are several, one
    of them nothing; None where the sequences fill the batch."""
    if not case.get("ragged"):
        return None
    n = torch.randint(1, case["seqlen"] + 1, (case["batch"],), generator=gen, device="cuda")
    n[0] = case["seqlen"]
    if case["batch"] > 2:
        n[1] = 0
    return n.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = torch.bfloat16 if case["dtype"] == BF16 else torch.float32

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    s = {"op": case["op"]}
    Bz = case["batch"]
    if case["op"].startswith("norm"):
        L, C = case["seqlen"], case["channels"]
        # channels of unequal size and place, as heads leave them; the gate lies in
        # the rows of the layer's first projection
        s["x"] = (normal(Bz, L, C, to=torch.float32) * torch.exp(0.5 * normal(C, to=torch.float32))
                  + 0.5 * normal(C, to=torch.float32)).to(dtype)
        s["gate"] = normal(Bz, L, 2 * C)[:, :, C:] if case["form"] != "plain" else None
        s["groups"], s["center"], s["gate_first"] = case["groups"], case["center"], case["form"] == "gate_first"
        s["weight"] = 1 + 0.2 * normal(C, to=torch.float32) if case["affine"] else None
        s["bias"] = normal(C, scale=0.1, to=torch.float32) if case["affine"] and case["center"] else None
        s["seqlens"] = _lengths(case, gen)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(Bz, L, C)
        return s
    H, K, Dk, Dv = case["heads"], case["kv_heads"], case["key"], case["value"]
    lead = (Bz,) if case["op"] == "attn_step" else (Bz, case["seqlen"])
    # queries, keys and values are parts of one projection's rows
    rows = normal(*lead, H * Dk + K * (Dk + Dv))
    s["q"] = rows[..., :H * Dk].unflatten(-1, (H, Dk))
    s["k"] = rows[..., H * Dk:(H + K) * Dk].unflatten(-1, (K, Dk))
    s["v"] = rows[..., (H + K) * Dk:].unflatten(-1, (K, Dv))
    # what a head keeps for 16 to 2048 steps, each moved a little
    spans = 16 * 128 ** (torch.arange(H, device="cuda") / max(H - 1, 1)) * torch.exp(0.1 * normal(H, to=torch.float32))
    s["log_decay"] = torch.log1p(-1 / spans)
    if case["op"] == "attn_step":
        s["state"] = normal(Bz, H, Dv, Dk, to=torch.float32)
        return s
    s["seqlens"] = _lengths(case, gen)
    s["initial_state"] = normal(Bz, H, Dv, Dk, to=torch.float32) if case["carry"] else None
    if case["op"] == "attn_bwd":
        s["dy"] = normal(*lead, H, Dv)
        s["dfinal_state"] = normal(Bz, H, Dv, Dk, to=torch.float32) if case["carry"] else None
    return s


def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    Bz = case["batch"]
    if case["op"].startswith("norm"):
        elements, gated = Bz * case["seqlen"] * case["channels"], case["form"] != "plain"
        params = 4 * case["channels"] * (1 + case["center"]) if case["affine"] else 0
        if case["op"] == "norm_fwd":
            return {"bytes": elements * (2 + gated) * es + params, "flops": elements * (8 + 5 * gated)}
        return {"bytes": elements * (3 + 2 * gated) * es + 2 * params, "flops": elements * (18 + 12 * gated)}
    H, K, Dk, Dv = case["heads"], case["kv_heads"], case["key"], case["value"]
    state, kv = Bz * H * Dk * Dv * 4, K * (Dk + Dv)
    if case["op"] == "attn_step":
        return {"bytes": 2 * state + Bz * (H * (Dk + Dv) + kv) * es, "flops": 5 * Bz * H * Dk * Dv}
    steps = Bz * case["seqlen"]
    if case["op"] == "attn_fwd":
        return {"bytes": steps * (H * (Dk + Dv) + kv) * es + state * (1 + case["carry"]),
                "flops": 4 * steps * H * Dk * Dv}
    return {"bytes": steps * (H * (2 * Dk + Dv) + 2 * kv) * es + state * (3 if case["carry"] else 0),
            "flops": 10 * steps * H * Dk * Dv}


# ---- the passes --------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import ssd_chunked_scan_chunk_amd as ssd

    op = s["op"]
    if op.startswith("norm"):
        form = dict(weight=s["weight"], bias=s["bias"], gate=s["gate"], eps=EPS, center=s["center"], silu=True,
                    gate_first=s["gate_first"], seqlens=s["seqlens"])
        if op == "norm_fwd":
            return {"y": ssd.group_norm_fwd(s["x"], s["groups"], **form)}
        return ssd.group_norm_bwd(s["x"], s["groups"], s["dy"], **form)
    args = [s[k] for k in ("q", "k", "v", "log_decay")]
    if op == "attn_step":
        return {"y": ssd.linear_attn_step(s["state"], *args), "state": s["state"]}
    if op == "attn_fwd":
        y, state = ssd.linear_attn_fwd(*args, initial_state=s["initial_state"], seqlens=s["seqlens"],
                                       return_final_state=True)
        return {"y": y, "state": state}
    return ssd.linear_attn_bwd(*args, s["dy"], initial_state=s["initial_state"], dfinal_state=s["dfinal_state"],
                               seqlens=s["seqlens"], return_dinitial_state=s["initial_state"] is not None)


def _plain(s):
    return {"attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step,
            "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[s["op"]](s)


def _valid(seqlens, L):
    """[batch, L] truth values: the steps that belong to the sequences."""
    return torch.arange(L, device=seqlens.device) < seqlens[:, None]


def _kept(seqlens, *rows):
    """The rows with those behind their sequence's end replaced by zeros."""
    if seqlens is None:
        return rows
    v = _valid(seqlens, rows[0].shape[1])
    return tuple(torch.where(v.view(v.shape + (1,) * (r.dim() - 2)), r, 0) for r in rows)


def _powers(log_decay, n):
    """e^(log_decay n) for whole numbers n, 0 where n is negative; [heads, ...]."""
    e = torch.exp(log_decay.double().view(-1, *(1,) * n.dim()) * n.clamp(min=0))
    return torch.where(n >= 0, e, 0).float()


SPAN = 128


def _heads_first(t, H, L):
    """[batch, L, heads, dim] -> [batch, heads, spans, SPAN, dim], fp32, zero
    rows at the end and heads repeated where they are shared."""
    t = torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, -L % SPAN)).transpose(1, 2)
    return t.repeat_interleave(H // t.shape[1], 1).unflatten(2, (-1, SPAN))


def _attend(q, k, v, log_decay, first, lead):
    """sum over j <= t of decay^(t-j) (q[t].k[j]) v[j] + decay^(t+lead) first q[t],
    on spans: inside each by its scores, across them by the states at their
    ends.  q, k, v as _heads_first gives them; first [batch, heads, value, key]."""
    n, at = q.shape[2], torch.arange(SPAN, device=q.device)
    within = _powers(log_decay, at[:, None] - at)[:, None]
    y = (q @ k.transpose(-1, -2) * within) @ v
    to_end = _powers(log_decay, SPAN - 1 - at)[:, None, :, None]
    ends = (v * to_end).transpose(-1, -2) @ k                               # [batch, heads, spans, value, key]
    spans = torch.arange(n, device=q.device)
    across = _powers(log_decay, (spans[:, None] - 1 - spans) * SPAN)        # span i reads the end of j < i
    entering = (across @ ends.flatten(3)).unflatten(3, ends.shape[3:])
    from_start = _powers(log_decay, at + 1)[:, None, :, None]
    y = y + (q @ entering.transpose(-1, -2)) * from_start
    if first is not None:
        reach = _powers(log_decay, spans[:, None] * SPAN + at + lead)[..., None]
        y = y + (q @ first[:, :, None].transpose(-1, -2)) * reach
    return y


def _last(k, v, log_decay, first, lens, more):
    """first decay^len + sum over j of decay^(len - 1 - j + more) v[j] k[j]^T, as
    [batch, heads, value, key]; rows behind the end are zero."""
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    to_end = lens[:, None] - 1 - torch.arange(k.shape[2], device=k.device)
    weight = torch.where(to_end >= 0, _powers(log_decay, to_end.clamp(min=0) + more), 0).transpose(0, 1)
    state = (v * weight[..., None]).transpose(-1, -2) @ k
    return state if first is None else state + first * _powers(log_decay, lens).t()[..., None, None]


def _lens(s):
    Bz, L = s["q"].shape[:2]
    return torch.full((Bz,), L, device="cuda") if s["seqlens"] is None else s["seqlens"].long()


def _rows(y, L, seqlens, dtype):
    y, = _kept(seqlens, y.flatten(2, 3)[:, :, :L].transpose(1, 2))
    return y.to(dtype).contiguous()


def _plain_attn_fwd(s):
    L, H, Dk = s["q"].shape[1:]
    q, k, v = (_heads_first(t, H, L) for t in _kept(s["seqlens"], s["q"], s["k"], s["v"]))
    y = _attend(q, k, v, s["log_decay"], s["initial_state"], 1) * Dk ** -0.5
    return {"y": _rows(y, L, s["seqlens"], s["v"].dtype),
            "state": _last(k, v, s["log_decay"], s["initial_state"], _lens(s), 0)}


def _plain_attn_bwd(s):
    L, H, Dk = s["q"].shape[1:]
    K, scale, decay, lens, dtype = s["k"].shape[2], Dk ** -0.5, s["log_decay"], _lens(s), s["q"].dtype
    kept = _kept(s["seqlens"], s["q"], s["k"], s["v"], s["dy"])
    q, k, v, dy = (_heads_first(t, H, L) for t in kept)
    first, last = s["initial_state"], s["dfinal_state"]
    flip = None if first is None else first.transpose(-1, -2)
    out = {"dq": _rows(_attend(dy, v, k, decay, flip, 1) * scale, L, s["seqlens"], dtype)}
    # the other two run from the sequences' ends: step t of the reversed rows is len - 1 - t
    turn = (lens[:, None] - 1 - torch.arange(L, device="cuda")).clamp(min=0)[:, :, None, None]
    back = [torch.take_along_dim(t, turn, 1) for t in kept]
    rq, rk, rv, rdy = (_heads_first(t, H, L) for t in _kept(s["seqlens"], *back))
    rq = rq * scale
    flip = None if last is None else last.transpose(-1, -2)
    dk, dv = _attend(rv, rdy, rq, decay, flip, 0), _attend(rk, rq, rdy, decay, last, 0)

    def turned(g):
        g = torch.take_along_dim(g.flatten(2, 3)[:, :, :L].transpose(1, 2), turn, 1)
        g, = _kept(s["seqlens"], g.unflatten(2, (K, H // K)).sum(3))
        return g.to(dtype)
    out.update(dk=turned(dk), dv=turned(dv),
               dinitial_state=_last(rq, rdy, decay, last, lens, 1) if first is not None else None)
    return out


def _plain_attn_step(s):
    H, Dk = s["q"].shape[1:]
    each = H // s["k"].shape[1]
    q, k, v = s["q"].float(), s["k"].float().repeat_interleave(each, 1), s["v"].float().repeat_interleave(each, 1)
    s["state"].copy_(s["state"] * torch.exp(s["log_decay"])[:, None, None] + v[..., None] * k[:, :, None])
    y = (s["state"] * q[:, :, None]).sum(-1) * Dk ** -0.5
    return {"y": y.to(s["v"].dtype), "state": s["state"]}


def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    g = torch.sigmoid(v)
    return g * (1 + v * (1 - g))


def _normed(s):
    """fp32 x, gate, the normalised rows and 1/sqrt(var + eps), by groups: [batch, seqlen, groups, channels]."""
    split = lambda t: None if t is None else t.unflatten(-1, (s["groups"], -1))  # noqa: E731
    x, = _kept(s["seqlens"], s["x"].float())
    gate = None if s["gate"] is None else _kept(s["seqlens"], s["gate"].float())[0]
    inner = x * _silu(gate) if s["gate_first"] else x
    inner = split(inner)
    if s["center"]:
        inner = inner - inner.mean(-1, keepdim=True)
    r = torch.rsqrt((inner * inner).mean(-1, keepdim=True) + EPS)
    return split(x), split(gate), inner * r, r, split(s["weight"]), split(s["bias"])


def _affine(n, weight, bias):
    p = n if weight is None else n * weight
    return p if bias is None else p + bias


def _plain_norm_fwd(s):
    _, gate, n, _, weight, bias = _normed(s)
    p = _affine(n, weight, bias)
    y = _silu(p) if gate is None else p if s["gate_first"] else p * _silu(gate)
    y, = _kept(s["seqlens"], y.flatten(2))
    return {"y": y.to(s["x"].dtype)}


def _plain_norm_bwd(s):
    x, gate, n, r, weight, bias = _normed(s)
    dtype = s["x"].dtype
    dy, = _kept(s["seqlens"], s["dy"].float())
    dy = dy.unflatten(-1, (s["groups"], -1))
    p, dgate = _affine(n, weight, bias), None
    if gate is None:
        dp = dy * _dsilu(p)
    elif s["gate_first"]:
        dp = dy
    else:
        dp, dgate = dy * _silu(gate), dy * p * _dsilu(gate)
    dn = dp if weight is None else dp * weight
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if s["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    dx = dx * r
    if s["gate_first"]:
        dx, dgate = dx * _silu(gate), dx * x * _dsilu(gate)
    dx, dgate = (None if t is None else _kept(s["seqlens"], t.flatten(2))[0].to(dtype) for t in (dx, dgate))
    return {"dx": dx, "dgate": dgate, "dweight": None if weight is None else (dp * n).sum((0, 1)).flatten(),
            "dbias": None if bias is None else dp.sum((0, 1)).flatten()}


# ---- the definitions in 64 bits --------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    H, each, scale = case["heads"], case["heads"] // case["kv_heads"], case["key"] ** -0.5
    decay = torch.exp(s["log_decay"])[:, None, None]
    q, k, v = s["q"], s["k"].repeat_interleave(each, -2), s["v"].repeat_interleave(each, -2)
    if case["op"] == "attn_step":
        S = decay * s["state"] + v[..., None] * k[..., None, :]
        return {"y": scale * (S @ q[..., None])[..., 0], "state": S}
    return _exact_attn(case, s, q, k, v, decay, scale, each)


def _exact_attn(case, s, q, k, v, decay, scale, each):
    """Step by step, forward for y and dq, backward for dk and dv."""
    Bz, L, H, Dk = q.shape
    Dv = v.shape[-1]
    lens = torch.full((Bz,), L, device="cuda") if s["seqlens"] is None else s["seqlens"].long()
    zero = q.new_zeros(Bz, H, Dv, Dk)
    back = case["op"] == "attn_bwd"
    S = zero if s["initial_state"] is None else s["initial_state"]
    out = torch.zeros_like(q) if back else torch.zeros_like(v)
    for t in range(L):
        live = (t < lens)[:, None, None]
        S = torch.where(live[..., None], decay * S + v[:, t, :, :, None] * k[:, t, :, None, :], S)
        if back:
            out[:, t] = live * scale * (s["dy"][:, t, :, None, :] @ S)[..., 0, :]
        else:
            out[:, t] = live * scale * (S @ q[:, t, :, :, None])[..., 0]
    if not back:
        return {"y": out, "state": S}
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    G = zero if s["dfinal_state"] is None else s["dfinal_state"]   # the adjoint of S[t], decay times that of S[t + 1]
    for t in reversed(range(L)):
        live = (t < lens)[:, None, None]
        full = G + scale * s["dy"][:, t, :, :, None] * q[:, t, :, None, :]
        dk[:, t] = live * (v[:, t, :, None, :] @ full)[..., 0, :]
        dv[:, t] = live * (full @ k[:, t, :, :, None])[..., 0]
        G = torch.where(live[..., None], decay * full, G)
    shared = lambda g: g.unflatten(2, (-1, each)).sum(3)  # noqa: E731
    return {"dq": out, "dk": shared(dk), "dv": shared(dv),
            "dinitial_state": G if s["initial_state"] is not None else None}


def _exact_norm(case, s):
    """Group by group and, for the gradients, by the Jacobian of the normalisation."""
    x, gate, C, G = s["x"], s["gate"], case["channels"], case["groups"]
    m, form = C // G, case["form"]
    live = torch.ones(x.shape[:2], device="cuda") if s["seqlens"] is None else _valid(s["seqlens"], x.shape[1])
    live = live[..., None].double()
    weight = x.new_ones(C) if s["weight"] is None else s["weight"]
    bias = x.new_zeros(C) if s["bias"] is None else s["bias"]
    sig = lambda t: 1 / (1 + torch.exp(-t))  # noqa: E731
    slope = lambda t: sig(t) + t * sig(t) * (1 - sig(t))  # noqa: E731
    back = case["op"] == "norm_bwd"
    y, dx, dgate = (torch.zeros_like(x) for _ in range(3))
    dweight, dbias = torch.zeros_like(weight), torch.zeros_like(bias)
    for g in range(G):
        c = slice(g * m, (g + 1) * m)
        xg, zg = x[..., c], None if gate is None else gate[..., c]
        u = xg * zg * sig(zg) if form == "gate_first" else xg
        if case["center"]:
            u = u - u.sum(-1, keepdim=True) / m
        sd = torch.sqrt((u ** 2).sum(-1, keepdim=True) / m + EPS)
        n = u / sd
        p = n * weight[c] + bias[c]
        if not back:
            y[..., c] = live * (p * sig(p) if form == "plain" else p * zg * sig(zg) if form == "gate" else p)
            continue
        d = live * s["dy"][..., c]
        if form == "plain":
            d = d * slope(p)
        elif form == "gate":
            dgate[..., c] = d * p * slope(zg)
            d = d * zg * sig(zg)
        dweight[c], dbias[c] = (d * n).sum((0, 1)), d.sum((0, 1))
        d = d * weight[c]
        du = (d - n * (d * n).sum(-1, keepdim=True) / m) / sd
        if case["center"]:
            du = du - du.sum(-1, keepdim=True) / m
        if form == "gate_first":
            dgate[..., c] = du * xg * slope(zg)
            du = du * zg * sig(zg)
        dx[..., c] = du
    if not back:
        return {"y": y}
    return {"dx": dx, "dgate": None if gate is None else dgate, "dweight": None if s["weight"] is None else dweight,
            "dbias": None if s["bias"] is None else dbias}
