"""GPU tests of linear attention with a decay for each head and of rotary positions against 64-bit
references (linattn_ref), alone and as a block runs them.  Every bound is the reference's, element
by element."""
import pytest
import torch

import linattn_ref as ref
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TD = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _columns(dev, *tensors, before=8, behind=16):
    """The tensors [b, L, n, w] as columns of one wider array, NaN before and behind them."""
    b, L = tensors[0].shape[:2]
    width = sum(t[0, 0].numel() for t in tensors)
    wide = torch.full((b, L, before + width + behind), float("nan"), device=dev, dtype=tensors[0].dtype)
    outs, at = [], before
    for t in tensors:
        n = t[0, 0].numel()
        wide[:, :, at:at + n] = t.reshape(b, L, n).to(dev)
        outs.append(wide[:, :, at:at + n].unflatten(2, t.shape[2:]))
        at += n
    return outs


def _inputs(dtype, b, L, G, H, dk, dv, dev, decay="token", state=True, seed=0, rate=0.3):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    td = TD[dtype]
    d = dict(zip("qkv", _columns(dev, rnd(b, L, G, dk).to(td), rnd(b, L, G, dk).to(td),
                                 rnd(b, L, H, dv).to(td))))
    d["g"] = None
    if decay == "head":
        d["g"] = (-rate * torch.rand(H, generator=gen)).to(dev)
    elif decay == "token":
        d["g"] = _columns(dev, (-rate * torch.rand(b, L, H, generator=gen) ** 3).to(td), before=1, behind=1)[0]
    d["h0"] = rnd(b, H, dv, dk).to(dev) if state else None
    return d


def _lengths(lengths, dev):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)


CASES = [
    # dtype, b, L, G, H, dk, dv, decay, state, lengths
    ("bf16", 1, 1, 1, 1, 8, 8, "token", True, None),
    ("fp32", 1, 1, 2, 2, 8, 8, "none", False, None),
    ("bf16", 2, 2, 1, 2, 16, 24, "token", False, None),
    ("fp32", 2, 17, 2, 2, 24, 16, "token", True, None),
    ("bf16", 1, 63, 2, 2, 64, 64, "token", True, None),
    ("bf16", 1, 64, 2, 2, 64, 64, "head", True, None),
    ("bf16", 1, 65, 2, 2, 64, 64, "none", True, None),
    ("fp32", 1, 65, 2, 2, 64, 64, "token", True, None),
    ("bf16", 2, 257, 2, 6, 72, 200, "token", True, None),
    ("fp32", 1, 257, 1, 3, 72, 200, "token", True, None),
    ("bf16", 1, 300, 4, 4, 128, 128, "token", False, None),
    ("fp32", 1, 200, 2, 2, 128, 128, "head", True, None),
    ("bf16", 1, 130, 1, 2, 136, 64, "token", True, None),
    ("bf16", 1, 150, 2, 2, 256, 256, "token", True, None),
    ("fp32", 1, 150, 1, 2, 256, 256, "token", True, None),
    ("bf16", 5, 140, 2, 4, 40, 72, "token", True, [140, 0, 1, 64, 65]),
    ("fp32", 4, 100, 1, 2, 64, 80, "head", True, [0, 100, 63, 99]),
    ("bf16", 3, 70, 2, 2, 32, 32, "none", False, [-5, 90, 33]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompts(case):
    dtype, b, L, G, H, dk, dv, decay, state, lengths = case
    dev = require_gpu()
    d = _inputs(dtype, b, L, G, H, dk, dv, dev, decay, state)
    scale = dk ** -0.5
    o, hT = ssd.ssd_linattn(**d, scale=scale, lengths=_lengths(lengths, dev))
    torch.cuda.synchronize()
    n = None if lengths is None else [min(max(m, 0), L) for m in lengths]
    ro, eo, rS, eS = ref.forward(**d, scale=scale, lengths=n)
    for i, m in enumerate(n or []):
        ro[i, m:], eo[i, m:] = 0, 0
    ref.check(o, ro, eo, "o")
    ref.check(hT, rS, eS, "hT")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decays_far_apart(dtype):
    """Decays of all sizes in one chunk: none, slow, some hundreds, minus infinity, and values
    above 0, which are taken as 0."""
    dev = require_gpu()
    d = _inputs(dtype, 2, 200, 2, 2, 64, 64, dev, seed=3)
    gen = torch.Generator().manual_seed(4)
    pick = torch.randint(0, 7, (2, 200, 2), generator=gen).to(dev)
    sizes = torch.tensor([0.0, -0.001, -1.0, -30.0, -300.0, -1e30, 2.0], device=dev).to(TD[dtype])
    d["g"] = sizes[pick]
    d["g"][0, 70] = -float("inf")
    d["g"][1, 0] = -float("inf")
    o, hT = ssd.ssd_linattn(**d)
    torch.cuda.synchronize()
    ro, eo, rS, eS = ref.forward(**d, scale=1.0)
    ref.check(o, ro, eo, "o")
    ref.check(hT, rS, eS, "hT")
    # nothing from before a token that forgets all
    late = {n: t[:, 70:] for n, t in d.items() if n in "qkvg"}
    r2, e2, rS, eS = ref.forward(**late, h0=torch.zeros_like(d["h0"]), scale=1.0)
    ref.check(o[:1, 70:], r2[:1], eo[:1, 70:] + e2[:1], "o behind it")


def test_a_nan_decay_reaches_only_what_follows():
    dev = require_gpu()
    d = _inputs("bf16", 1, 200, 1, 2, 64, 64, dev, seed=6)
    clean, _ = ssd.ssd_linattn(**d)
    d["g"] = d["g"].clone()
    d["g"][0, 100, 1] = float("nan")
    o, hT = ssd.ssd_linattn(**d)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :, 0], clean[:, :, 0]) and torch.equal(o[0, :100, 1], clean[0, :100, 1])
    assert o[0, 100:, 1].isnan().all() and hT[0, 1].isnan().all() and not hT[0, 0].isnan().any()


@pytest.mark.parametrize("dtype,L", [("bf16", 190), ("fp32", 64), ("bf16", 2000)])
def test_a_prompt_in_parts(dtype, L):
    """The final state continues a prompt, in its own buffer too; o and hT given by the caller."""
    dev = require_gpu()
    d = _inputs(dtype, 2, L, 2, 4, 64, 72, dev, seed=7)
    whole, hT = ssd.ssd_linattn(**d)
    cut = L // 3
    first = {n: (t[:, :cut].contiguous() if n in "qkvg" else t) for n, t in d.items()}
    rest = {n: t[:, cut:].contiguous() for n, t in d.items() if n in "qkvg"}
    o1, h = ssd.ssd_linattn(**first)
    given = torch.full_like(rest["v"], float("nan"))
    o2, h2 = ssd.ssd_linattn(**rest, h0=h, o=given, hT=h)
    torch.cuda.synchronize()
    assert o2 is given and h2 is h
    o = torch.cat([o1, o2], 1).float()
    # two roundings of the state and scores in other chunks: 2^-8 of the largest output each
    tol = 4 * 2.0 ** -8 if dtype == "bf16" else 1e-5
    assert (o - whole.float()).abs().max() <= tol * whole.float().abs().max()
    assert (h - hT).abs().max() <= 1e-5 * hT.abs().max()


def test_rows_behind_a_sequence():
    """Left as they were in a given output, zero in an allocated one, and not read."""
    dev = require_gpu()
    lengths = [130, 0, 64, 3]
    d = _inputs("bf16", 4, 130, 2, 2, 64, 40, dev, seed=8)
    lt = _lengths(lengths, dev)
    for n in "qkvg":
        d[n] = d[n].clone()
    clean, h1 = ssd.ssd_linattn(**d, lengths=lt)
    for i, m in enumerate(lengths):
        for n in "qkvg":
            d[n][i, m:] = float("nan")
    given = torch.full_like(clean, 7.0)
    o, h2 = ssd.ssd_linattn(**d, lengths=lt, o=given)
    torch.cuda.synchronize()
    for i, m in enumerate(lengths):
        assert torch.equal(o[i, :m], clean[i, :m])
        assert (o[i, m:] == 7).all() and (clean[i, m:] == 0).all()
    assert torch.equal(h1, h2) and torch.equal(h1[1], d["h0"][1])


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def _grad_inputs(dtype, b, L, G, H, dk, dv, dev, decay, state, seed=20):
    d = _inputs(dtype, b, L, G, H, dk, dv, dev, decay, state, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    d["do"] = _columns(dev, torch.randn(b, L, H, dv, generator=gen).to(TD[dtype]))[0]
    d["dhT"] = torch.randn(b, H, dv, dk, generator=gen).to(dev) if state else None
    return d


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients(case):
    dtype, b, L, G, H, dk, dv, decay, state, lengths = case
    dev = require_gpu()
    d = _grad_inputs(dtype, b, L, G, H, dk, dv, dev, decay, state)
    got = ssd.ssd_linattn_backward(**d, scale=dk ** -0.5, lengths=_lengths(lengths, dev))
    torch.cuda.synchronize()
    n = None if lengths is None else [min(max(m, 0), L) for m in lengths]
    want = ref.backward(**d, scale=dk ** -0.5, lengths=n)
    for name, x, (r, e) in zip(("dq", "dk", "dv", "dg", "dh0"), got, want):
        if x is None:
            assert name == "dg" and decay != "token" or name == "dh0" and not state
            continue
        if name != "dh0":
            for i, m in enumerate(n or []):
                r[i, m:], e[i, m:] = 0, 0
        ref.check(x, r, e, name)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_of_decays_far_apart(dtype):
    dev = require_gpu()
    d = _grad_inputs(dtype, 2, 200, 2, 2, 64, 64, dev, "token", True)
    gen = torch.Generator().manual_seed(4)
    pick = torch.randint(0, 7, (2, 200, 2), generator=gen).to(dev)
    sizes = torch.tensor([0.0, -0.001, -1.0, -30.0, -300.0, -1e30, 2.0], device=dev).to(TD[dtype])
    d["g"] = sizes[pick]
    d["g"][0, 70] = -float("inf")
    got = ssd.ssd_linattn_backward(**d)
    torch.cuda.synchronize()
    want = ref.backward(**d, scale=1.0)
    off = ((d["g"] > 0) | (d["g"] < -1000)).cpu()
    want[3][0][off], want[3][1][off] = 0, 0
    for name, x, (r, e) in zip(("dq", "dk", "dv", "dg", "dh0"), got, want):
        ref.check(x, r, e, name)


def test_gradients_match_differences():
    """The forward call itself along random directions: fp32 values, summed in 64 bits."""
    dev = require_gpu()
    d = _grad_inputs("fp32", 1, 150, 1, 2, 16, 24, dev, "token", True)
    d["g"] = (d["g"] - 0.01).contiguous()
    do, dhT = d.pop("do"), d.pop("dhT")
    grads = ssd.ssd_linattn_backward(do, **d, dhT=dhT, scale=0.25)

    def value(args):
        o, hT = ssd.ssd_linattn(**args, scale=0.25)
        return ((o.double() * do).sum() + (hT.double() * dhT).sum()).item()

    gen = torch.Generator().manual_seed(9)
    for name, grad in zip(("q", "k", "v", "g", "h0"), grads):
        x = d[name].contiguous()
        step = torch.randn(x.shape, generator=gen).to(dev) * (2.0 ** -10 if name != "g" else 2.0 ** -12)
        up, down = x + step, x - step
        slope = value({**d, name: up}) - value({**d, name: down})
        # what the values really moved by; third-order terms and fp32's sums: 1e-3 of the size
        along = (grad.double() * (up.double() - down.double()))
        assert abs(slope - along.sum().item()) <= 1e-3 * along.norm().item() + 1e-4 * abs(slope)


def test_gradients_behind_a_sequence():
    dev = require_gpu()
    lengths = [130, 0, 64, 3]
    d = _grad_inputs("bf16", 4, 130, 2, 4, 64, 40, dev, "token", True)
    lt = _lengths(lengths, dev)
    for n in ("q", "k", "v", "g", "do"):
        d[n] = d[n].clone()
    clean = ssd.ssd_linattn_backward(**d, lengths=lt)
    for i, m in enumerate(lengths):
        for n in ("q", "k", "v", "g", "do"):
            d[n][i, m:] = float("nan")
    given = {n: torch.full_like(t, 7.0) for n, t in zip(("dq", "dk", "dv", "dg", "dh0"), clean)}
    got = ssd.ssd_linattn_backward(**d, lengths=lt, **given)
    torch.cuda.synchronize()
    for x, y, name in zip(got, clean, given):
        assert x is given[name]
        for i, m in enumerate(lengths):
            if name == "dh0":
                assert torch.equal(x, y) and torch.equal(x[1], d["dhT"][1])
            else:
                assert torch.equal(x[i, :m], y[i, :m])
                assert (x[i, m:] == 7).all() and (y[i, m:] == 0).all()


# ---------------------------------------------------------------------------
# single tokens
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("case", [
    ("bf16", 1, 1, 1, 8, 8, "token"), ("fp32", 3, 2, 2, 16, 24, "token"), ("bf16", 2, 2, 4, 24, 16, "head"),
    ("bf16", 4, 1, 3, 40, 72, "token"), ("fp32", 2, 2, 2, 64, 64, "none"), ("bf16", 3, 2, 2, 128, 128, "token"),
    ("fp32", 2, 1, 2, 72, 200, "token"), ("bf16", 2, 2, 2, 136, 8, "token"), ("bf16", 2, 1, 2, 256, 256, "token"),
    ("fp32", 1, 1, 1, 8, 256, "head")], ids=str)
def test_step(case):
    dtype, b, G, H, dk, dv, decay = case
    dev = require_gpu()
    d = _inputs(dtype, b, 1, G, H, dk, dv, dev, decay)
    row = {n: (t[:, 0] if t is not None and t.dim() > 1 else t) for n, t in d.items() if n in "qkvg"}
    h = d["h0"].clone()
    ro, eo, rS, eS = ref.step(row["q"], row["k"], row["v"], row["g"], h, dk ** -0.5)
    o = ssd.ssd_linattn_step(row["q"], row["k"], row["v"], h, row["g"], scale=dk ** -0.5)
    torch.cuda.synchronize()
    ref.check(o, ro, eo, "o")
    ref.check(h, rS, eS, "h")


def test_step_decays():
    dev = require_gpu()
    d = _inputs("fp32", 2, 1, 1, 4, 32, 32, dev)
    g = torch.tensor([[-float("inf"), 0.0, 3.0, -200.0], [-1e30, -0.1, -90.0, float("nan")]], device=dev)
    h = d["h0"].clone()
    q, k, v = (d[n][:, 0] for n in "qkv")
    ssd.ssd_linattn_step(q, k, v, h, g)
    torch.cuda.synchronize()
    kv = v[..., None] * k.repeat_interleave(4, 1)[:, :, None, :]
    assert torch.equal(h[0, 0], kv[0, 0]) and torch.equal(h[1, 0], kv[1, 0])
    # a decay of exactly 1: one rounding, of h + v k (exact in 64 bits but for its own sum's 2^-53)
    exact = d["h0"][0, 2].double() + v[0, 2].double()[:, None] * k[0, 0].double()[None]
    assert ((h[0, 2].double() - exact).abs() <= ref.U * (1 + 1e-6) * exact.abs()).all()
    assert h[1, 3].isnan().all() and not h[:, :3].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_continue_a_prompt(dtype):
    """A plan bound once, its tensors refilled token by token, and o in v's own buffer."""
    dev = require_gpu()
    d = _inputs(dtype, 3, 80, 2, 4, 64, 48, dev, seed=9)
    whole, hT = ssd.ssd_linattn(**d)
    first = {n: (t[:, :70].contiguous() if n in "qkvg" else t) for n, t in d.items()}
    _, h = ssd.ssd_linattn(**first)
    rows = {n: d[n][:, 0].contiguous() for n in "qkvg"}
    plan = ssd.LinattnStepPlan(rows["q"], rows["k"], rows["v"], h, rows["g"], o=rows["v"])
    outs = []
    for t in range(70, 80):
        for n in "qkvg":
            rows[n].copy_(d[n][:, t])
        outs.append(plan.run().clone())
    torch.cuda.synchronize()
    o = torch.stack(outs, 1).float()
    w = whole[:, 70:].float()
    tol = 4 * 2.0 ** -8 if dtype == "bf16" else 1e-5
    assert (o - w).abs().max() <= tol * w.abs().max()
    assert (h - hT).abs().max() <= 1e-5 * hT.abs().max()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
ROTARY = [
    # dtype, b, L, heads, groups, width, rotated, interleaved, inverse, positions, scale
    ("bf16", 1, 1, 1, 0, 2, 2, False, False, "start", 1.0),
    ("fp32", 2, 3, 2, 1, 6, 4, True, False, "first", 1.0),
    ("bf16", 2, 5, 3, 1, 7, 6, True, True, "each", 1.0),
    ("bf16", 1, 9, 3, 2, 33, 32, False, False, "each", 0.5),
    ("bf16", 2, 33, 4, 2, 64, 64, False, False, "first", 1.0),
    ("bf16", 2, 33, 4, 2, 64, 64, True, True, "first", 1.0),
    ("fp32", 2, 33, 4, 4, 64, 32, False, True, "each", 1.25),
    ("fp32", 3, 70, 3, 1, 100, 36, True, True, "each", 1.0),
    ("bf16", 1, 40, 2, 2, 80, 48, False, False, "start", 1.0),
    ("bf16", 1, 40, 2, 2, 80, 24, False, False, "start", 1.0),
    ("bf16", 1, 4, 1, 1, 4096, 4096, False, False, "first", 1.0),
    ("fp32", 1, 4, 1, 1, 4096, 4094, True, False, "first", 1.0),
    ("bf16", 2, 2500, 2, 1, 128, 128, False, False, "first", 1.0),
    ("bf16", 1, 9000, 2, 0, 64, 32, True, False, "start", 1.0),
]


@pytest.mark.parametrize("case", ROTARY, ids=str)
def test_rotary(case):
    dtype, b, L, hq, hk, w, rot, inter, inverse, mode, scale = case
    dev = require_gpu()
    gen = torch.Generator().manual_seed(L + w)
    rnd = lambda n: torch.randn(b, L, n, w, generator=gen).to(TD[dtype])
    xs = _columns(dev, *[rnd(n) for n in (hq, hk) if n], before=3 if w % 2 else 8)
    freqs = ssd.rotary_frequencies(rot, device=dev)
    t = torch.arange(L, dtype=torch.int32)
    given = {"start": None, "first": torch.randint(-5, 1 << 20, (b,), generator=gen, dtype=torch.int32),
             "each": torch.randint(-(1 << 31), (1 << 31) - 1, (b, L), generator=gen, dtype=torch.int32)}[mode]
    at = t.expand(b, L) if given is None else given[:, None] + t if mode == "first" else given
    ys = ssd.ssd_rotary(xs[0], xs[1] if hk else None, freqs, None if given is None else given.to(dev),
                        interleaved=inter, inverse=inverse, scale=scale)
    torch.cuda.synchronize()
    for x, y in zip(xs, ys if hk else [ys]):
        r, e = ref.rotary(x, freqs, at, inter, inverse, scale)
        ref.check(y, r, e, "rotated")
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_single_tokens_in_place_and_back(inter):
    dev = require_gpu()
    gen = torch.Generator().manual_seed(2)
    q, k = (torch.randn(37, n, 64, generator=gen).to(dev) for n in (4, 1))
    at = torch.randint(0, 1 << 20, (37,), generator=gen, dtype=torch.int32).to(dev)
    freqs = ssd.rotary_frequencies(48, device=dev)
    long, _ = ssd.ssd_rotary(q[:, None], k[:, None], freqs, at, interleaved=inter)
    q1, k1 = q.clone(), k.clone()
    a, b = ssd.ssd_rotary(q1, k1, freqs, at, interleaved=inter, q_out=q1, k_out=k1)
    torch.cuda.synchronize()
    assert a is q1 and b is k1 and torch.equal(q1, long[:, 0]) and not torch.equal(q1, q)
    ssd.ssd_rotary(q1, k1, freqs, at, interleaved=inter, inverse=True, q_out=q1, k_out=k1)
    torch.cuda.synchronize()
    assert (q1 - q).abs().max() < 1e-5 and (k1 - k).abs().max() < 1e-5
