"""Linear attention with a decay for each head, its gradients and rotary positions in 64 bits, with
the rounding errors that the kernels may make.

Functions return (value, bound) pairs: bound holds, element by element, what is lost on the way
(before the output's own rounding).  The kernels go chunk by chunk (64 tokens), so with the
pairs (t, s) of a target and a source, D the decay between them, S the state before a chunk,

* bf16 only: scores of pairs within a chunk, and the elements of the state that a chunk reads, are
  rounded to bf16 once (half a step, 2^-8 of the value); nothing else is.
* a sum of n terms in any order: n U times the sum of their absolute values (U = 2^-24).  An
  output's terms go through a sum over keys (n = width), one over the tokens of a chunk, and for
  each chunk in between one product and one sum; the state's through three parts a token.
* a factor exp(G): the logarithm's base 2 (a rounded constant and a rounded product, 2 U |G|
  together), sums of the rests of 2^-8 (below 2^-27 ln 2, less than U), exp2 itself (2 U) and the
  products with it.
"""
import torch

U = 2.0 ** -24
HALF = 2.0 ** -8
CHUNK = 64
NOTHING = 1e-35         # factors below fp32's normal numbers are taken as zero


def per_head(t, heads):
    """[b, L, n, w] -> [b, H, L, w] in 64 bits."""
    t = t.detach().cpu().double()
    return t.repeat_interleave(heads // t.shape[2], 2).transpose(1, 2)


def log_decays(g, b, L, H, lengths):
    """[b, H, L] log decays, at most 0 (one that forgets all as -1e4), 0 behind each sequence."""
    if g is None:
        d = torch.zeros(b, H, L, dtype=torch.float64)
    elif g.dim() == 1:
        d = g.detach().cpu().double()[None, :, None].repeat(b, 1, L)
    else:
        d = g.detach().cpu().double().transpose(1, 2).clone()
    d = d.clamp(-1e4, 0)
    for i, n in enumerate(lengths or []):
        d[i, :, n:] = 0
    return d


def clear(t, lengths):
    """[b, H, L, w]: zero behind each sequence."""
    t = t.clone()
    for i, n in enumerate(lengths or []):
        t[i, :, n:] = 0
    return t


class Pairs:
    """Decays between targets t and sources s <= t (back in time: s >= t), [b, H, t, s]."""

    def __init__(self, d, back=False):
        L = d.shape[2]
        self.G = G = d.cumsum(2)
        gap = (G[..., None, :] - G[..., :, None]) if back else (G[..., :, None] - G[..., None, :])
        keep = torch.ones(L, L, dtype=torch.bool).tril()
        keep = keep.T if back else keep
        self.D = torch.where(keep, gap, torch.tensor(-float("inf"), dtype=torch.float64)).exp()
        self.size = torch.where(keep, gap, torch.zeros((), dtype=torch.float64)).abs()
        # from the first state (back in time: the last one) to each target
        self.far = (G[..., -1:] - G) if back else G
        c = torch.arange(L) // CHUNK
        self.same = (c[:, None] == c[None, :]) & keep
        self.chunks = int(c[-1]) + 1
        self.back = back


def states(k, v, first, p):
    """[b, H, chunk, dv, dk]: the state before each chunk (back in time: behind it)."""
    L, out = k.shape[2], []
    for c in range(p.chunks):
        if p.back:
            t = min((c + 1) * CHUNK, L)              # sources from t on, decayed to the end of t - 1
            w = (p.G[..., t:] - p.G[..., t - 1:t]).exp()
            s, f, far = slice(t, L), w, (p.G[..., -1] - p.G[..., t - 1]).exp()
        else:
            t = c * CHUNK
            if t == 0:
                s, f, far = slice(0, 0), p.G[..., :0], torch.ones_like(p.G[..., 0])
            else:
                s, f, far = slice(0, t), (p.G[..., t - 1:t] - p.G[..., :t]).exp(), p.G[..., t - 1].exp()
        S = torch.matmul((v[:, :, s] * f[..., None]).transpose(2, 3), k[:, :, s])
        if first is not None:
            S = S + far[..., None, None] * first
        out.append(S)
    return torch.stack(out, 2)


def walk(q, k, v, d, first, scale, bf16, back=False):
    """Outputs [b, H, L, dv] of queries against states, and what may be lost."""
    p = Pairs(d, back)
    score = torch.matmul(q, k.transpose(2, 3)) * p.D * scale
    o = torch.matmul(score, v)
    sizes = torch.matmul(q.abs(), k.abs().transpose(2, 3)) * p.D * abs(scale)
    A = torch.matmul(sizes, v.abs())
    E = torch.matmul(sizes * p.size, v.abs())
    if first is not None:
        far = p.far.exp()[..., None] * scale
        o = o + torch.matmul(q, first.transpose(2, 3)) * far
        a = torch.matmul(q.abs(), first.abs().transpose(2, 3)) * far.abs()
        A, E = A + a, E + a * p.far.abs()[..., None]
    bound = U * ((q.shape[3] + CHUNK + 4 * p.chunks + 16) * A + 2 * E) + NOTHING
    if bf16:
        bound = bound + HALF * torch.matmul(score.abs() * p.same, v.abs())
        S = states(k, v, first, p).abs()
        for c in range(p.chunks):
            t = slice(c * CHUNK, min((c + 1) * CHUNK, q.shape[2]))
            last = p.G[..., t.stop - 1:t.stop]
            before = p.G[..., t.start - 1:t.start] if c > 0 else 0.0
            far = (last - p.G[..., t]) if back else (p.G[..., t] - before)
            r = torch.matmul(q[:, :, t].abs(), S[:, :, c].transpose(2, 3))
            bound[:, :, t] += HALF * (1 + HALF) * abs(scale) * r * far.exp()[..., None]
        bound = bound * (1 + HALF)
    return o, bound


def last_state(k, v, d, first, weight=1.0, back=False):
    """The state behind all tokens (back in time: before them) [b, H, dv, dk] and its bound."""
    G = d.cumsum(2)
    far = G if back else G[..., -1:] - G
    w = far.exp() * weight
    S = torch.matmul((v * w[..., None]).transpose(2, 3), k)
    A = torch.matmul((v * w[..., None]).abs().transpose(2, 3), k.abs())
    E = torch.matmul((v * (w * far)[..., None]).abs().transpose(2, 3), k.abs())
    if first is not None:
        all_ = G[..., -1].exp()[..., None, None]
        S, A = S + all_ * first, A + all_ * first.abs()
        E = E + all_ * first.abs() * G[..., -1].abs()[..., None, None]
    chunks = (k.shape[2] + CHUNK - 1) // CHUNK
    return S, U * ((3 * CHUNK + 4 * chunks + 16) * A + 2 * E) + NOTHING


def forward(q, k, v, g, h0, scale, lengths=None):
    """(o [b, L, H, dv], bound, hT, bound)."""
    b, L, H, _ = v.shape
    bf16 = q.dtype == torch.bfloat16
    d = log_decays(g, b, L, H, lengths)
    q, k, v = (clear(per_head(t, H), lengths) for t in (q, k, v))
    first = None if h0 is None else h0.detach().cpu().double()
    o, eo = walk(q, k, v, d, first, scale, bf16)
    S, eS = last_state(k, v, d, first)
    return o.transpose(1, 2), eo.transpose(1, 2), S, eS


def backward(do, q, k, v, g, h0, dhT, scale, lengths=None):
    """[(value, bound)] of dq, dk [b, L, G, dk], dv [b, L, H, dv], dg [b, L, H] and dh0."""
    b, L, H, _ = v.shape
    G, bf16 = q.shape[2], q.dtype == torch.bfloat16
    d = log_decays(g, b, L, H, lengths)
    do, q, k, v = (clear(per_head(t, H), lengths) for t in (do, q, k, v))
    first = None if h0 is None else h0.detach().cpu().double()
    last = None if dhT is None else dhT.detach().cpu().double()
    T = lambda s: None if s is None else s.transpose(2, 3)
    # the backward state is kept with the scale in it: what is read from it has none
    raw = lambda s: None if s is None else s / scale
    dq = walk(do, v, k, d, T(first), scale, bf16)
    dk = walk(v, do, q, d, raw(T(last)), scale, bf16, back=True)
    dv = walk(k, q, do, d, raw(last), scale, bf16, back=True)
    dh0 = last_state(q, do, d, last, weight=scale, back=True)
    half = HALF if bf16 else 0.0

    # g_t scales every product of a read at i >= t with a write at j < t
    p = Pairs(d)
    reads = torch.matmul(do, v.transpose(2, 3)) * p.D * scale             # [.., i, j]
    pairs = torch.matmul(q, k.transpose(2, 3)) * reads
    sizes = torch.matmul(q.abs(), k.abs().transpose(2, 3)) * p.D * abs(scale)
    sizes = sizes * torch.matmul(do.abs(), v.abs().transpose(2, 3))
    S, dS = states(k, v, first, p), states(q, do * scale, last, Pairs(d, True))
    t = torch.arange(L)
    over = (t[:, None] >= t[None, :]).double()                             # [t', t]: t' >= t
    def passing(m):
        # sum over i >= t > j of m[i, j]
        less = (t[:, None] < t[None, :]).double()                          # [j, t]: j < t
        return (torch.matmul(m.transpose(2, 3), over) * less).sum(2)
    dg, A, E = passing(pairs), passing(sizes), passing(sizes * p.size)
    if first is not None:
        far = p.G.exp() * scale
        u = (torch.matmul(q, T(first)) * do).sum(3) * far
        a = (torch.matmul(q.abs(), T(first).abs()) * do.abs()).sum(3) * far.abs()
        dg, A, E = dg + torch.matmul(u, over), A + torch.matmul(a, over), E + torch.matmul(a * p.G.abs(), over)
    if last is not None:
        behind = p.G[..., -1:] - p.G
        w = (torch.matmul(k, T(last)) * v).sum(3) * behind.exp()
        a = (torch.matmul(k.abs(), T(last).abs()) * v.abs()).sum(3) * behind.exp()
        less = 1.0 - over
        dg, A, E = dg + torch.matmul(w, less), A + torch.matmul(a, less), E + torch.matmul(a * behind.abs(), less)
        if first is not None:
            x, a = (first * last).sum((2, 3)), (first * last).abs().sum((2, 3))
            all_ = p.G[..., -1].exp()
            dg = dg + (x * all_)[..., None]
            A, E = A + (a * all_)[..., None], E + (a * all_ * p.G[..., -1].abs())[..., None]
    # in each chunk the pairs are summed by targets and by sources, which cancel where both lie on
    # the same side of t
    chunk = torch.matmul(sizes * p.same, torch.ones(L, 1, dtype=torch.float64)).squeeze(3)
    inside = torch.zeros_like(chunk)
    for c in range(p.chunks):
        s = slice(c * CHUNK, min((c + 1) * CHUNK, L))
        inside[..., s] = chunk[..., s].sum(2, keepdim=True)
    n = q.shape[3] + v.shape[3] + 2 * CHUNK + 4 * p.chunks + 32
    bound = U * (n * (A + 2 * inside) + 2 * E) + NOTHING
    if bf16:
        # the scores of pairs within a chunk, rounded once, the same in q . dq and in k . dk: half a
        # step of each product that passes t, and nothing of one that does not
        bound = bound + HALF * passing(pairs.abs() * p.same)
        # reads and writes of rounded states, and rounded states against their gradients
        for c in range(p.chunks):
            s = slice(c * CHUNK, min((c + 1) * CHUNK, L))
            before = p.G[..., s.start - 1:s.start] if c > 0 else 0.0
            at, whole = p.G[..., s] - before, p.G[..., s.stop - 1:s.stop] - before
            eu = (torch.matmul(q[:, :, s].abs(), T(S[:, :, c]).abs()) * do[:, :, s].abs()).sum(3)
            ew = (torch.matmul(k[:, :, s].abs(), T(dS[:, :, c]).abs()) * v[:, :, s].abs()).sum(3)
            eu, ew = eu * at.exp() * abs(scale), ew * (whole - at).exp()
            m = s.stop - s.start
            up = over[:m, :m]
            ex = (S[:, :, c] * dS[:, :, c]).abs().sum((2, 3))[..., None] * whole.exp()
            bound[..., s] += half * (1 + half) * (torch.matmul(eu, up) + torch.matmul(ew, 1.0 - up) + ex)
    by_group = lambda pair: tuple(x.transpose(1, 2).unflatten(2, (G, H // G)).sum(3) for x in pair)
    heads = lambda pair: tuple(x.transpose(1, 2) for x in pair)
    dg_pair = (dg.transpose(1, 2), bound.transpose(1, 2))
    return [by_group(dq), by_group(dk), heads(dv), dg_pair, dh0]


def step(q, k, v, g, h, scale):
    """(o [b, H, dv], bound, h, bound) of one token."""
    row = lambda t: t[:, None]
    o, _, S, _ = forward(row(q), row(k), row(v), g if g is None or g.dim() == 1 else row(g), h, scale)
    a = log_decays(g if g is None or g.dim() == 1 else row(g), v.shape[0], 1, v.shape[1], None)
    size = h.detach().cpu().double().abs() * a.exp()[..., None]
    kk = per_head(row(k), v.shape[1]).abs()
    size = size + v.detach().cpu().double().abs()[..., None] * kk
    eS = U * (6 + 2 * a.abs()[..., None]) * size + NOTHING
    qq = per_head(row(q), v.shape[1]).abs()
    eo = ((eS + (q.shape[-1] + 2) * U * size) * qq).sum(3) * abs(scale)
    return o[:, 0], eo, S, eS


def check(out, ref, bound, what, dtype=None):
    """|out - ref| <= bound + half a step of the output's type, element by element."""
    dtype = dtype or out.dtype
    half = U if dtype == torch.float32 else HALF
    o = out.detach().cpu().double()
    assert o.shape == ref.shape, (what, o.shape, ref.shape)
    tol = bound + (ref.abs() + bound) * half
    bad = ~((o - ref).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off; first {i}: "
                             f"{o[i]} for {ref[i]} (allowed {tol[i]:.3e})")
    worst = ((o - ref).abs() / tol).max().item() if o.numel() else 0.0
    print(f"  {what}: worst error {worst:.3f} of the bound", flush=True)


def rotary(x, freqs, positions, interleaved, inverse, scale):
    """x [b, L, n, w], positions [b, L] -> (value, bound): the sines are off by the eighth of a
    turn's rounding, the polynomial's few, the scale's and the products': 8 U of each term."""
    x, f = x.detach().cpu().double(), freqs.detach().cpu().double()
    half = f.numel()
    angle = positions.detach().cpu().double()[:, :, None, None] * f
    if inverse:
        angle = -angle
    j = torch.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    y, e = x.clone(), torch.zeros_like(x)
    y[..., a] = scale * (x[..., a] * angle.cos() - x[..., b] * angle.sin())
    y[..., b] = scale * (x[..., b] * angle.cos() + x[..., a] * angle.sin())
    size = abs(scale) * (x[..., a].abs() + x[..., b].abs())
    e[..., a] = e[..., b] = 8 * U * size
    return y, e
