"""The decays' gradient of linear attention in 64 bits, part by part, with the standard deviation of
the kernels' rounding errors.

The bound of linattn_ref.backward adds up the largest error of every product, which for random inputs
is about as large as the gradient itself.  Here errors are independent, each uniform within its half
step h (variance h^2 / 3), so that variances add up; a sum of such errors passes eight standard
deviations with a probability below 2 exp(-32).  With V the sum of the squares of an element's products:

* bf16 only: the states that the two walks hand over are rounded once, each element by its own half
  step; scores, states that are read and what is added to a state go in as two parts, which leaves
  2^-16 of each of the three.
* sums in fp32: partial sums of products of random signs are sqrt(V) in size, and each of n additions
  rounds one, by U at most: U sqrt(n / 3 V).  The pairs of a chunk are added up by targets and by
  sources, where those on one side of the token cancel: their squares count twice in V.
* factors exp(G): (3 + 2 |G|) U of each product (two roundings of the logarithm, exp2, a product).
* the output's own rounding is not random here: half a step of its value at most.
"""
import torch

import linattn_ref as ref

SIGMAS = 8.0
TWO_PARTS = 2.0 ** -16


def _half_steps(x, bits):
    """Half a step of numbers of `bits` bits at x."""
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - bits - 1) * (x != 0)


def decay_gradient(do, q, k, v, g, h0, dhT, scale, lengths=None):
    """(parts, deviation): the gradient's four parts [b, L, H], whose sum it is, by name, and the
    standard deviation of the error before the output's rounding."""
    b, L, H, _ = v.shape
    bf16 = q.dtype == torch.bfloat16
    d = ref.log_decays(g, b, L, H, lengths)
    n = q.shape[3] + v.shape[3] + 2 * ref.CHUNK + 4 * ((L + ref.CHUNK - 1) // ref.CHUNK) + 32
    do, q, k, v = (ref.clear(ref.per_head(t, H), lengths) for t in (do, q, k, v))
    T = lambda s: s.transpose(2, 3)
    p = ref.Pairs(d)
    first, last = (None if t is None else t.detach().cpu().double() for t in (h0, dhT))
    S, dS = ref.states(k, v, first, p), ref.states(q, do * scale, last, ref.Pairs(d, True))
    parts = {name: torch.zeros(b, H, L, dtype=torch.float64) for name in ("inside", "read", "written", "cross")}
    var = torch.zeros(b, H, L, dtype=torch.float64)
    for c in range(p.chunks):
        s = slice(c * ref.CHUNK, min((c + 1) * ref.CHUNK, L))
        m = s.stop - s.start
        before = p.G[..., s.start - 1:s.start] if c > 0 else 0.0
        at, whole = p.G[..., s] - before, p.G[..., s.stop - 1:s.stop] - before
        Q, K, V, O, D = q[:, :, s], k[:, :, s], v[:, :, s], do[:, :, s], p.D[:, :, s, s] * scale
        t = torch.arange(m)
        upto = (t[:, None] >= t[None, :]).double()          # [i, t]: i >= t
        less = 1.0 - upto                                   # [j, t]: j < t
        passing = lambda x: (torch.matmul(T(x), upto) * less).sum(2)
        pairs = torch.matmul(Q, T(K)) * torch.matmul(O, T(V)) * D
        squares = torch.matmul(Q ** 2, T(K ** 2)) * torch.matmul(O ** 2, T(V ** 2)) * D ** 2
        Sc, dSc = S[:, :, c], dS[:, :, c]
        reads = (torch.matmul(Q, T(Sc)) * O).sum(3) * at.exp() * scale
        reads2 = (torch.matmul(Q ** 2, T(Sc ** 2)) * O ** 2).sum(3) * (at.exp() * scale) ** 2
        left = whole - at
        writes = (torch.matmul(K, T(dSc)) * V).sum(3) * left.exp()
        writes2 = (torch.matmul(K ** 2, T(dSc ** 2)) * V ** 2).sum(3) * left.exp() ** 2
        parts["inside"][..., s] = passing(pairs)
        parts["read"][..., s] = torch.matmul(reads, upto)
        parts["written"][..., s] = torch.matmul(writes, less)
        parts["cross"][..., s] = (Sc * dSc).sum((2, 3))[..., None] * whole.exp()
        cross2 = ((Sc * dSc) ** 2).sum((2, 3))[..., None] * whole.exp() ** 2
        size = passing(squares) + torch.matmul(reads2, upto) + torch.matmul(writes2, less) + cross2
        twice = 2 * squares.sum((2, 3))[..., None]
        of_factors = (passing(squares * (3 + 2 * p.size[:, :, s, s]) ** 2)
                      + torch.matmul(reads2 * (3 - 2 * at) ** 2, upto)
                      + torch.matmul(writes2 * (3 - 2 * left) ** 2, less) + cross2 * (3 - 2 * whole) ** 2)
        x = ref.U ** 2 * (n / 3 * (size + twice) + of_factors)
        if bf16:
            x = x + 3 * TWO_PARTS ** 2 / 3 * (size + twice)
            x = x + ((_half_steps(Sc, 8) * dSc) ** 2).sum((2, 3))[..., None] / 3 * whole.exp() ** 2
        var[..., s] = x
    out = lambda t: ref.clear(t[..., None], lengths)[..., 0].transpose(1, 2)
    return {name: out(t) for name, t in parts.items()}, out(var).sqrt()


def misses(x, value, deviation, dtype):
    """Which elements of x are further from value than eight deviations and half a step allow."""
    half = ref.U if dtype == torch.float32 else ref.HALF
    off = SIGMAS * deviation + ref.NOTHING
    return ~((x.detach().cpu().double() - value).abs() <= off + half * (value.abs() + off))


def check(x, value, deviation, what):
    assert x.shape == value.shape, what
    bad = misses(x, value, deviation, x.dtype)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements off"


def one_rounding(x, value):
    """The error's 2-norm over that of one rounding to bf16 (uniform within each value's half step)."""
    expected = (_half_steps(value, 8) ** 2 / 3).sum().sqrt()
    return ((x.detach().cpu().double() - value).norm() / expected).item()
