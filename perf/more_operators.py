"""Linear attention with a decay for each head, as it is measured: prompts, their gradients,
single tokens, and the rotary positions of its queries and keys.

`run` computes a case in plain torch (`own` false) or through the library (`own` true).  Heads
are those of this repository's workloads (4 to 32 heads, 64 to 256 wide, shared over groups as B
and C are), its lengths (256 tokens in fp32, 2K, 16K), decode batches of 1 and 128, and odd or
ragged ones between them.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
_CHUNK = 64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the short fp32 problem: few heads, four chunks, one launch's latency
        dict(name="linattn fp32 256 tokens", op="linattn", dtype="fp32", batch=1, seqlen=256,
             heads=4, groups=4, key=64, value=64, decay="token", state=False, ragged=False),
        # a 16K-token prompt with a decay per token, continued from a state, q, k and v columns
        # of one projection
        dict(name="linattn bf16 16K tokens", op="linattn", dtype="bf16", batch=1, seqlen=16384,
             heads=16, groups=16, key=128, value=128, decay="token", state=True, ragged=False),
        # prompts of 2K tokens whose value heads share queries and keys, as x does B and C
        dict(name="linattn bf16 shared keys", op="linattn", dtype="bf16", batch=2, seqlen=2048,
             heads=24, groups=4, key=128, value=64, decay="token", state=False, ragged=False),
        # a padded batch of unlike lengths, odd widths, one fixed decay per head
        dict(name="linattn bf16 ragged odd", op="linattn", dtype="bf16", batch=5, seqlen=2500,
             heads=6, groups=6, key=72, value=200, decay="head", state=True, ragged=True),
        # gradients of the short fp32 problem
        dict(name="gradient fp32 256 tokens", op="backward", dtype="fp32", batch=1, seqlen=256,
             heads=4, groups=4, key=64, value=64, decay="token", state=True, ragged=False),
        # gradients of a training batch
        dict(name="gradient bf16 4x4K tokens", op="backward", dtype="bf16", batch=4, seqlen=4096,
             heads=16, groups=16, key=128, value=128, decay="token", state=False, ragged=False),
        # gradients of a padded batch with shared queries and keys and of a given first state
        dict(name="gradient bf16 ragged shared", op="backward", dtype="bf16", batch=3, seqlen=1501,
             heads=12, groups=4, key=96, value=64, decay="token", state=True, ragged=True),
        # one token of one sequence, and of a full decode batch
        dict(name="step bf16 b1", op="step", dtype="bf16", batch=1, seqlen=1, heads=16, groups=16,
             key=128, value=128, decay="token", state=True, ragged=False),
        dict(name="step bf16 b128", op="step", dtype="bf16", batch=128, seqlen=1, heads=16,
             groups=16, key=128, value=128, decay="token", state=True, ragged=False),
        # queries and keys of a 16K-token prompt, rotated in halves
        dict(name="rotary bf16 16K tokens", op="rotary", dtype="bf16", batch=1, seqlen=16384,
             heads=16, groups=16, width=128, rotated=128, interleaved=False, each=False, step=False,
             inverse=False, far=0),
        # the gradient of a padded batch's rotation: interleaved pairs, part of an odd head, far
        # positions given token by token
        dict(name="rotary fp32 part interleaved", op="rotary", dtype="fp32", batch=3, seqlen=700,
             heads=12, groups=2, width=100, rotated=36, interleaved=True, each=True, step=False,
             inverse=True, far=1 << 20),
        # one token of each sequence of a decode batch
        dict(name="rotary step bf16 b128", op="rotary", dtype="bf16", batch=128, seqlen=1, heads=16,
             groups=16, width=128, rotated=128, interleaved=False, each=False, step=True,
             inverse=False, far=100000),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linattn", "linattn", "backward", "backward", "step", "rotary"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    groups = _log_int(rng, 1, 16)
    heads = groups * rng.choice([1, 1, 1, 2, 4])
    if op == "rotary":
        width = 2 * _log_int(rng, 16, 128)
        rotated = width if rng.random() < 0.5 else 2 * rng.randint(1, width // 2)
        step = rng.random() < 0.3
        batch = _log_int(rng, 1, 256) if step else rng.choice([1, 2, 3, 8])
        most = (1 << (25 if case["dtype"] == "bf16" else 24)) // (batch * (heads + groups) * width)
        case.update(batch=batch, seqlen=1 if step else _log_int(rng, 1, max(1, min(32768, most))),
                    heads=heads, groups=groups, width=width, rotated=rotated,
                    interleaved=rng.random() < 0.5, each=not step and rng.random() < 0.5,
                    step=step, inverse=rng.random() < 0.5,
                    far=rng.choice([0, 0, 5000, 100000, 1 << 20]))
        return case
    key, value = 8 * _log_int(rng, 2, 32), 8 * _log_int(rng, 2, 32)
    if op == "step":
        batch = min(_log_int(rng, 1, 256), max(1, (1 << 25) // (heads * key * value)))
    else:
        batch = rng.choice([1, 1, 2, 3, 8])
    # values of the widest input, and products of the states
    most = (1 << 25) if case["dtype"] == "bf16" else (1 << 22)
    most = min(most // max(key, value), (1 << 32) // (key * value)) // (batch * heads)
    if op == "backward":
        most //= 2
    seqlen = 1 if op == "step" else _log_int(rng, 1, max(1, min(32768, most)))
    case.update(batch=batch, seqlen=seqlen, heads=heads, groups=groups, key=key, value=value,
                decay=rng.choice(["token", "token", "token", "head", "none"]),
                state=op == "step" or rng.random() < 0.5,
                ragged=op != "step" and rng.random() < 0.4)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kw = {"generator": g, "device": "cuda"}
    td = _TYPES[case["dtype"]]
    b, L, H, G = case["batch"], case["seqlen"], case["heads"], case["groups"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, **kw) * scale

    state = {"case": case}
    if case["op"] == "rotary":
        w, rot = case["width"], case["rotated"]
        # queries and keys are columns of one projection's output
        both = normal(b, L, (H + G) * w).to(td)
        state["q"] = both[:, :, :H * w].unflatten(2, (H, w))
        state["k"] = both[:, :, H * w:].unflatten(2, (G, w))
        state["freqs"] = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").float() / rot)
        # each sequence's first position, or every token's own (a packed batch begins anew)
        first = (torch.rand(b, **kw) * case["far"]).to(torch.int32)
        state["positions"] = first
        if case["each"]:
            t = torch.arange(L, device="cuda", dtype=torch.int32) % (L // 2 + 1)
            state["positions"] = first[:, None] + t
        if case["step"]:
            state["q"], state["k"] = state["q"][:, 0], state["k"][:, 0]
        return state
    dk, dv = case["key"], case["value"]
    # q, k and v are columns of one projection's output
    both = normal(b, L, 2 * G * dk + H * dv).to(td)
    state["q"] = both[:, :, :G * dk].unflatten(2, (G, dk))
    state["k"] = both[:, :, G * dk:2 * G * dk].unflatten(2, (G, dk))
    state["v"] = both[:, :, 2 * G * dk:].unflatten(2, (H, dv))
    # heads that forget within a few tokens to ones that keep about a thousand
    rate = -torch.exp(math.log(0.001) + torch.linspace(0, 1, H, device="cuda") * math.log(400.0))
    state["g"] = None
    if case["decay"] == "head":
        state["g"] = rate
    elif case["decay"] == "token":
        state["g"] = (rate * 2 * torch.rand(b, L, H, **kw)).to(td)
    state["h"] = normal(b, H, dv, dk) if case["state"] else None
    state["lengths"] = None
    if case["ragged"]:
        # a padded batch: from empty to full rows, one of them full
        n = (torch.rand(b, **kw) * (L + 1)).to(torch.int32)
        n[0] = L
        state["lengths"] = n
    if case["op"] == "backward":
        state["do"] = normal(b, L, H, dv).to(td)
        state["dhT"] = normal(b, H, dv, dk, scale=0.1) if case["state"] else None
    if case["op"] == "step":
        # a decode loop's tensors hold one token per sequence
        for name in ("q", "k", "v"):
            state[name] = state[name][:, 0]
        if case["decay"] == "token":
            state["g"] = state["g"][:, 0]
        if own:
            # it binds them once and calls the plan for every token
            import state_space_sequence_cumsum_amd as ssd
            state["plan"] = ssd.LinattnStepPlan(state["q"], state["k"], state["v"], state["h"],
                                                state["g"], scale=_scale(case))
    return state


def _scale(case):
    return case["key"] ** -0.5


# ---------------------------------------------------------------------------
# plain forms: 32 bits throughout (sums of decays and angles in 64), rounded once at the end
# ---------------------------------------------------------------------------
def _decays(state):
    """Log decays [b, L, H] in 64 bits."""
    case, g = state["case"], state["g"]
    shape = case["batch"], case["seqlen"], case["heads"]
    if g is None:
        return torch.zeros(shape, device="cuda", dtype=torch.float64)
    return g.double().expand(shape) if g.dim() == 1 else g.double()


def _behind(t, lengths):
    """Zero in the rows behind each sequence's length."""
    if lengths is None:
        return t
    keep = torch.arange(t.shape[1], device=t.device)[None, :] < lengths[:, None]
    return t.masked_fill(~keep.view(*keep.shape, *[1] * (t.dim() - 2)), 0)


def _chunks(t, heads):
    """[b, L, n, w] or [b, L, n] -> [b, heads, chunks, 64, w] in 32 bits ([..., 64] in 64)."""
    b, L = t.shape[:2]
    pad = -L % _CHUNK
    if t.dim() == 3:
        t = torch.nn.functional.pad(t, (0, 0, 0, pad))
        return t.unflatten(1, (-1, _CHUNK)).permute(0, 3, 1, 2)
    t = torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, pad))
    t = t.repeat_interleave(heads // t.shape[2], 2)
    return t.unflatten(1, (-1, _CHUNK)).permute(0, 3, 1, 2, 4)


def _tokens(t, L, dtype, lengths, groups=None):
    """[b, H, chunks, 64, w] -> [b, L, H, w] (heads of a group added up)."""
    t = t.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :L]
    if groups is not None:
        t = t.unflatten(2, (groups, -1)).sum(3)
    return _behind(t.to(dtype), lengths).contiguous()


class _Decay:
    """Factors of the chunks: within one, from its start, to its end, and between chunks."""

    def __init__(self, g):
        sums = g.cumsum(-1)                                              # [b, H, chunks, 64]
        total = sums[..., -1]
        self.start = sums.exp().float()[..., None]
        self.end = (total[..., None] - sums).exp().float()[..., None]
        self.whole = total.exp().float()
        lower = torch.ones(_CHUNK, _CHUNK, device=g.device, dtype=torch.bool).tril()
        gap = (sums[..., :, None] - sums[..., None, :]).masked_fill(~lower, -math.inf)
        self.inner = gap.exp().float()                                   # [.., target, source]
        # state before chunk i from what chunk j < i adds: the decay of the chunks between
        ends = total.cumsum(-1)
        n = ends.shape[-1]
        gap = (ends - total)[..., :, None] - ends[..., None, :]
        earlier = torch.ones(n, n, device=g.device, dtype=torch.bool).tril(-1)
        self.between = gap.masked_fill(~earlier, -math.inf).exp().float()
        self.before = (ends - total).exp().float()[..., None, None]      # from the first state
        self.after = (ends[..., -1:] - ends).exp().float()[..., None, None]   # to the last one
        self.all = ends[..., -1].exp().float()[..., None, None]


def _states(added, d, first):
    """States [b, H, chunks, dk, dv] before each chunk, and the last one."""
    s = torch.matmul(d.between, added.flatten(3)).view_as(added)
    last = (added * d.after).sum(2)
    if first is not None:
        s = s + d.before * first[:, :, None]
        last = last + d.all * first
    return s, last


def _plain_forward(state):
    case, lengths = state["case"], state["lengths"]
    L, H, td = case["seqlen"], case["heads"], state["q"].dtype
    d = _Decay(_chunks(_behind(_decays(state), lengths), H))
    q = _chunks(state["q"], H)
    k, v = (_chunks(_behind(state[n], lengths), H) for n in ("k", "v"))
    first = None if state["h"] is None else state["h"].transpose(2, 3)
    s, last = _states(torch.matmul((k * d.end).transpose(3, 4), v), d, first)
    o = torch.matmul(torch.matmul(q, k.transpose(3, 4)) * d.inner, v)
    o = (o + torch.matmul(q, s) * d.start) * _scale(case)
    return _tokens(o, L, td, lengths), last.transpose(2, 3).contiguous()


def _plain_backward(state):
    case, lengths = state["case"], state["lengths"]
    L, H, G, td = case["seqlen"], case["heads"], case["groups"], state["q"].dtype
    scale = _scale(case)
    d = _Decay(_chunks(_behind(_decays(state), lengths), H))
    q, k, v, do = (_chunks(_behind(state[n], lengths), H) for n in ("q", "k", "v", "do"))
    first = None if state["h"] is None else state["h"].transpose(2, 3)
    last = None if state["dhT"] is None else state["dhT"].transpose(2, 3)
    s, _ = _states(torch.matmul((k * d.end).transpose(3, 4), v), d, first)
    # gradients of the state behind each chunk, and of the first one
    added = torch.matmul((q * d.start).transpose(3, 4), do) * scale
    ds = torch.matmul(d.between.transpose(2, 3), added.flatten(3)).view_as(added)
    dfirst = (added * d.before).sum(2)
    if last is not None:
        ds = ds + d.after * last[:, :, None]
        dfirst = dfirst + d.all * last
    a = torch.matmul(q, k.transpose(3, 4)) * d.inner * scale             # [.., target, source]
    c = torch.matmul(do, v.transpose(3, 4)) * d.inner * scale
    qs = torch.matmul(do, s.transpose(3, 4)) * (d.start * scale)
    ks = torch.matmul(v, ds.transpose(3, 4)) * d.end
    dq = torch.matmul(c, k) + qs
    dk = torch.matmul(c.transpose(3, 4), q) + ks
    dv = torch.matmul(a.transpose(3, 4), do) + torch.matmul(k, ds) * d.end
    dg = None
    if case["decay"] == "token":
        pairs = torch.matmul(q, k.transpose(3, 4)) * c
        later = (pairs.sum(4) - pairs.sum(3) + (q * qs).sum(4)).flip(3).cumsum(3).flip(3)
        k_part = (k * ks).sum(4)
        dg = later + k_part.cumsum(3) - k_part + ((s * ds).sum((3, 4)) * d.whole)[..., None]
        dg = _behind(dg.permute(0, 2, 3, 1).flatten(1, 2)[:, :L].to(td), lengths).contiguous()
    return [_tokens(dq, L, td, lengths, G), _tokens(dk, L, td, lengths, G),
            _tokens(dv, L, td, lengths), dg,
            None if first is None else dfirst.transpose(2, 3).contiguous()]


def _plain_step(state):
    case = state["case"]
    H, td = case["heads"], state["q"].dtype
    q, k = (state[n].float().repeat_interleave(H // case["groups"], 1) for n in ("q", "k"))
    a = 1.0 if state["g"] is None else torch.exp(state["g"].float())[..., None, None]
    state["h"].mul_(a).add_(state["v"].float()[..., None] * k[:, :, None, :])
    o = (state["h"] * q[:, :, None, :]).sum(-1) * _scale(case)
    return o.to(td), state["h"]


def _plain_rotary(state):
    case = state["case"]
    rot, td = case["rotated"], state["q"].dtype
    pos = state["positions"]
    if pos.dim() == 1 and not case["step"]:
        pos = pos[:, None] + torch.arange(case["seqlen"], device=pos.device)
    angle = pos.double()[..., None, None] * state["freqs"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if case["inverse"]:
        sin = -sin

    def turn(x):
        r, rest = x[..., :rot].float(), x[..., rot:]
        if case["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r.to(td), rest], -1)

    return turn(state["q"]), turn(state["k"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        plain = {"linattn": _plain_forward, "backward": _plain_backward, "step": _plain_step,
                 "rotary": _plain_rotary}
        return plain[op](state)

    import state_space_sequence_cumsum_amd as ssd
    if op == "linattn":
        return ssd.ssd_linattn(state["q"], state["k"], state["v"], state["g"], state["h"],
                               scale=_scale(case), lengths=state["lengths"])
    if op == "backward":
        return list(ssd.ssd_linattn_backward(state["do"], state["q"], state["k"], state["v"],
                                             state["g"], state["h"], state["dhT"],
                                             scale=_scale(case), lengths=state["lengths"]))
    if op == "step":
        return state["plan"].run(), state["h"]
    return ssd.ssd_rotary(state["q"], state["k"], state["freqs"], state["positions"],
                          interleaved=case["interleaved"], inverse=case["inverse"])


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    b, L, H, G = case["batch"], case["seqlen"], case["heads"], case["groups"]
    if case["op"] == "rotary":
        n = b * L * (H + G) * case["width"]
        return {"bytes": 2 * n * e + 4 * b, "flops": 3 * n * case["rotated"] // case["width"]}
    dk, dv = case["key"], case["value"]
    if case["ragged"]:
        # one full sequence, the others half as long on average
        L = L * (b + 1) / (2 * b)
    states = 4 * b * H * dk * dv
    gates = e * b * L * H if case["decay"] == "token" else 4 * H
    if case["op"] == "step":
        return {"bytes": 2 * states + e * b * (2 * G * dk + 2 * H * dv) + gates,
                "flops": 5 * b * H * dk * dv}
    tokens = b * L * e
    # the recurrence's own products: the state's update and what is read from it
    if case["op"] == "linattn":
        return {"bytes": tokens * (2 * G * dk + 2 * H * dv) + gates
                + states * (2 if case["state"] else 1),
                "flops": 4 * b * L * H * dk * dv}
    # q, k, v, do, g and their gradients; states: the first, its gradient, the last one's
    return {"bytes": tokens * (4 * G * dk + 3 * H * dv) + 2 * gates
            + states * (3 if case["state"] else 0),
            "flops": 10 * b * L * H * dk * dv}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        w, rot, L = case["width"], case["rotated"], case["seqlen"]
        f, outs = state["freqs"].double(), []
        for x in (state["q"], state["k"]):
            x = x.double().reshape(case["batch"], L, -1, w)
            pos = state["positions"].double().view(case["batch"], -1)
            if pos.shape[1] != L:
                pos = pos + torch.arange(L, device=x.device)
            turn = torch.polar(torch.ones(1, device=x.device, dtype=torch.float64),
                               pos[:, :, None] * f)[:, :, None]
            if case["inverse"]:
                turn = turn.conj()
            even = torch.arange(rot // 2, device=x.device) * (2 if case["interleaved"] else 1)
            odd = even + (1 if case["interleaved"] else rot // 2)
            z = torch.complex(x[..., even], x[..., odd]) * turn
            y = x.clone()
            y[..., even], y[..., odd] = z.real, z.imag
            outs.append(y[:, 0] if case["step"] else y)
        return tuple(outs)
    b, L, H, G = case["batch"], case["seqlen"], case["heads"], case["groups"]
    if L > 20000:
        return None
    step, backward = case["op"] == "step", case["op"] == "backward"
    n = torch.full((b,), L, device="cuda") if state["lengths"] is None else state["lengths"].long()

    def rows(t):
        # [L, b, H, w], zero behind each sequence
        t = (t[:, None] if step else t).double()
        t = torch.stack([t[:, :, h * t.shape[2] // H] for h in range(H)], 2)
        for i, m in enumerate(n.tolist()):
            t[i, m:] = 0
        return t.transpose(0, 1).contiguous()

    q, k, v = rows(state["q"]), rows(state["k"]), rows(state["v"])
    a = torch.ones(L, b, H, 1, 1, device="cuda", dtype=torch.float64)
    if state["g"] is not None:
        g = state["g"].double()
        g = g.expand(b, L, H) if g.dim() == 1 else g.view(b, L, H)
        a = g.exp().transpose(0, 1)[..., None, None].contiguous()
        for i, m in enumerate(n.tolist()):
            a[m:, i] = 1
    S = torch.zeros(b, H, case["value"], case["key"], device="cuda", dtype=torch.float64)
    if state["h"] is not None:
        S = S + state["h"]
    scale = 1.0 / math.sqrt(case["key"])
    do = rows(state["do"]) if backward else None
    outs = []
    for t in range(L):
        S = a[t] * S + v[t, :, :, :, None] * k[t, :, :, None, :]
        if backward:
            outs.append((do[t, :, :, :, None] * S).sum(2))               # dq of each head
        else:
            outs.append((S * q[t, :, :, None, :]).sum(3))
    outs = torch.stack(outs) * scale                                     # [L, b, H, w]
    for i, m in enumerate(n.tolist()):
        outs[m:, i] = 0
    if step:
        return outs[0], S
    if not backward:
        return outs.transpose(0, 1), S
    dhT = torch.zeros_like(S) if state["dhT"] is None else state["dhT"].double()
    dS = dhT.clone()
    dks, dvs = [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        dS = dS + scale * do[t, :, :, :, None] * q[t, :, :, None, :]
        dks[t] = (dS * v[t, :, :, :, None]).sum(2)
        dvs[t] = (dS * k[t, :, :, None, :]).sum(3)
        dS = dS * a[t]
    dk, dv = torch.stack(dks), torch.stack(dvs)
    for i, m in enumerate(n.tolist()):
        dk[m:, i] = 0
        dv[m:, i] = 0
    dg = None
    if case["decay"] == "token":
        # what a decay scales: all that is read behind it less what is written behind it
        dg = ((q * outs).sum(3) - (k * dk).sum(3)).flip(0).cumsum(0).flip(0)
        dg = dg + (dhT * S).sum((2, 3))
        for i, m in enumerate(n.tolist()):
            dg[m:, i] = 0
        dg = dg.transpose(0, 1)
    shared = lambda t: t.transpose(0, 1).unflatten(2, (G, H // G)).sum(3)    # noqa: E731
    return [shared(outs), shared(dk), dv.transpose(0, 1), dg,
            dS if state["h"] is not None else None]
