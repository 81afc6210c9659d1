"""The operators around the forward in 64 bits, with the rounding errors fp32 kernels may make.

Each function returns (value, bound): bound holds, element by element, what 32-bit arithmetic
may lose on the way (before the output's own rounding), from the terms themselves:

* U = 2^-24 is half a step of fp32, one rounding; a hardware exp2 or reciprocal is taken as
  off by at most 2 U relative (one step).
* exp2 of a rounded argument a: relative error U |a| ln 2 * (roundings of a) + 2 U.
* a sum of n terms in any order: n U times the sum of their absolute values.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def d64(t):
    return None if t is None else t.detach().cpu().double()


def silu(v, ev):
    """(silu(v), error) for v off by ev: |silu'| <= 1.1; the sigmoid's exp2 has a rounded
    product and constant as its argument (2 U |v|), the sum, reciprocal and product three more."""
    s = torch.sigmoid(v)
    y = v * s
    return y, 1.1 * ev + y.abs() * ((1 - s) * (2 * v.abs() + 2) + 4) * U


def softplus(v, ev):
    """log(1 + exp(v)): slope at most 1; exp2's argument, the quotient s (three roundings and a
    reciprocal), the polynomial (4.1e-9 < U, its own roundings below 2 U) and the sum."""
    y = torch.logaddexp(v, torch.zeros_like(v))
    tail = torch.log1p(torch.exp(-v.abs()))
    return y, ev * torch.sigmoid(v) + tail * (2 * v.abs() + 12) * U + y * U


def check(out, ref, bound, what, dtype=None):
    """Element by element: |out - ref| <= bound + half a step of the output's type (and a
    subnormal's step, 2^-126, for flushed results); an infinite bound allows any value."""
    dtype = dtype or out.dtype
    o = d64(out)
    assert o.shape == ref.shape, (what, o.shape, ref.shape)
    tol = bound + (ref.abs() + bound) * HALF_STEP[dtype] + 2.0 ** -126
    bad = ~((o - ref).abs() <= tol) & ~torch.isinf(bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off; first {i}: "
                             f"{o[i]} for {ref[i]} (allowed {tol[i]:.3e})")
    share = ((o - ref).abs() / tol)[~torch.isinf(bound)]
    worst = share.max().item() if share.numel() else 0.0
    print(f"  {what}: worst error {worst:.3f} of the bound", flush=True)


def conv(x, weight, bias, state, lengths, act):
    """x [b, L, c], state [b, K-1, c] or None, lengths list or None -> (y, bound, final)."""
    x, w, bias, state = d64(x), d64(weight), d64(bias), d64(state)
    b, L, c = x.shape
    k = w.shape[1]
    if state is None:
        state = torch.zeros(b, k - 1, c, dtype=torch.float64)
    full = torch.cat([state, x], 1)
    v = torch.zeros(b, L, c, dtype=torch.float64) + (0 if bias is None else bias)
    size = v.abs()
    for j in range(k):
        term = full[:, j:j + L] * w[:, j]
        v, size = v + term, size + term.abs()
    ev = (k + 1) * U * size
    y, ey = silu(v, ev) if act else (v, ev)
    final = torch.stack([full[i, n:n + k - 1] for i, n in enumerate(lengths or [L] * b)])
    return y, ey, final


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None, act=False, run=None):
    """x, dt, z [b, L, c]; B, C [b, L, G, N] -> (y, bound, hT, bound).  run: the most roundings
    that a sum of steps goes through where tokens are split into runs (None: L).

    Negative step sizes grow a state exponentially.  Once the magnitude of a state, or of the
    terms of an output, passes 2^127, fp32 cannot hold it (its largest value is 2^128 - 2^104):
    the bound of what depends on it is infinite from there on."""
    x, d, A, B, C = d64(x), d64(dt), d64(A), d64(B), d64(C)
    D, z, dt_bias, h0 = d64(D), d64(z), d64(dt_bias), d64(h0)
    b, L, c = x.shape
    N = A.shape[1]
    rep = lambda t: t.repeat_interleave(c // t.shape[2], 2)
    B, C = rep(B), rep(C)
    ed = torch.zeros_like(d)
    if dt_bias is not None:
        d = d + dt_bias
        ed = U * d.abs()
    if act:
        d, ed = softplus(d, ed)
    n = torch.tensor(lengths if lengths is not None else [L] * b)
    h = torch.zeros(b, c, N, dtype=torch.float64) if h0 is None else h0.clone()
    size, eh = h.abs(), torch.zeros_like(h)
    y = torch.zeros(b, L, c, dtype=torch.float64)
    ey = torch.zeros_like(y)
    over = torch.zeros(b, c, N, dtype=torch.bool)
    inf, most = float("inf"), 2.0 ** 127
    for t in range(L):
        dv, xv = d[:, t, :, None], x[:, t, :, None]
        rate = (dv * A).abs()
        a = torch.exp(dv * A)
        # the exponent: A log2(e) and its product with d rounded (3 U with the constant), d
        # itself off by ed; where tokens are split into runs, exp of a run's summed steps
        # carries the sum's error, at most L (or run) U of it, in place of the single steps'
        ea = rate * (3 + (L if run is None else run)) * U + ed[:, t, :, None] * A.abs() + 2 * U
        term = dv * xv * B[:, t]
        et = term.abs() * 2 * U + ed[:, t, :, None] * (xv * B[:, t]).abs()
        new = a * h + term
        nsize = a * size + term.abs()
        neh = a * eh + ea * a * size + et + 2 * U * nsize
        on = (t < n)[:, None, None]
        h, size, eh = (torch.where(on, p, q) for p, q in ((new, h), (nsize, size), (neh, eh)))
        over = over | (size > most)
        y[:, t] = (C[:, t] * h).sum(-1)
        e = (C[:, t].abs() * (eh + (N + 2) * U * size)).sum(-1)
        far = over.any(-1) | ((C[:, t].abs() * size).sum(-1) > most)
        ey[:, t] = torch.where(far, inf, e)
    if D is not None:
        y, ey = y + D * x, ey + 2 * U * (D * x).abs()
    ey = ey + U * y.abs()
    if z is not None:
        g, eg = silu(z, torch.zeros_like(z))
        y, ey = y * g, ey * (g.abs() + eg) + y.abs() * eg + U * (y * g).abs()
    return y, ey, h, torch.where(over, inf, eh)


def norm(x, weight, z=None, residual=None, ngroups=1, eps=1e-5, scale=1.0, gate_after=False):
    """[rows, c] -> (y, bound, sum, bound)."""
    v, w, z, residual = d64(x), d64(weight), d64(z), d64(residual)
    ev = torch.zeros_like(v)
    g = None
    if z is not None:
        g, eg = silu(z, torch.zeros_like(z))
    if g is not None and not gate_after:
        v, ev = v * g, v.abs() * eg + U * (v * g).abs()
    if residual is not None:
        s = float(torch.tensor(scale, dtype=torch.float32))
        v, ev = residual + s * v, abs(s) * ev + U * ((s * v).abs() + (residual + s * v).abs())
    vg, eg_ = v.unflatten(1, (ngroups, -1)), ev.unflatten(1, (ngroups, -1))
    cg = vg.shape[-1]
    e = float(torch.tensor(eps, dtype=torch.float32))
    ss = vg.square().sum(-1, keepdim=True)
    r = torch.rsqrt(ss / cg + e)
    # the sum of squares, its mean, the root and the reciprocal
    er = (vg.abs() * eg_).sum(-1, keepdim=True) / (ss + cg * e) + (cg + 10) * U
    y = (vg * r).flatten(1) * w
    ey = (eg_ * r).flatten(1) * w.abs() + y.abs() * (er.expand_as(vg).flatten(1) + 3 * U)
    if g is not None and gate_after:
        y, ey = y * g, ey * (g.abs() + eg) + y.abs() * eg + U * (y * g).abs()
    return y, ey, v, ev
