"""GPU tests of linear attention and rotary positions as a program runs them: prompts of many
segments, repeated, captured and simultaneous calls, given workspaces and streams, and a block."""
import pytest
import torch

import linattn_ref as ref
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu
from test_gpu_linattn import TD, _columns, _grad_inputs, _inputs, _lengths

pytestmark = pytest.mark.gpu

GRADS = ("dq", "dk", "dv", "dg", "dh0")

LONG = [
    # dtype, b, L, G, H, dk, dv, decay, state, lengths
    ("bf16", 1, 320, 1, 1, 64, 64, "token", True, None),
    ("bf16", 1, 321, 1, 1, 64, 64, "token", False, None),
    ("fp32", 1, 256, 1, 1, 64, 64, "token", True, None),
    ("fp32", 1, 193, 2, 2, 40, 136, "token", True, None),
    ("bf16", 1, 1100, 1, 2, 128, 128, "token", True, None),
    ("bf16", 1, 1024, 1, 2, 256, 200, "none", True, None),
    ("fp32", 1, 700, 1, 2, 128, 64, "head", True, None),
    ("fp32", 1, 520, 1, 1, 256, 256, "token", True, None),
    ("bf16", 4, 900, 1, 2, 72, 136, "token", True, [900, 0, 65, 320]),
    ("fp32", 3, 600, 1, 2, 64, 48, "token", False, [1, 600, 449]),
]


def _cleared(pairs, lengths, upto):
    for r, e in pairs:
        for i, m in enumerate(lengths or []):
            if i < upto:
                r[i, m:], e[i, m:] = 0, 0


@pytest.mark.parametrize("case", LONG, ids=str)
def test_prompts_of_many_segments(case):
    dtype, b, L, G, H, dk, dv, decay, state, lengths = case
    dev = require_gpu()
    # slow decays: what the first tokens leave reaches the last ones
    d = _inputs(dtype, b, L, G, H, dk, dv, dev, decay, state, seed=30, rate=0.02)
    prob = ssd.linattn_problem(d["q"], d["v"])
    assert ssd.ssd_linattn_workspace_bytes(prob) > 1, "one walk: no segments"
    o, hT = ssd.ssd_linattn(**d, scale=dk ** -0.5, lengths=_lengths(lengths, dev))
    torch.cuda.synchronize()
    ro, eo, rS, eS = ref.forward(**d, scale=dk ** -0.5, lengths=lengths)
    _cleared([(ro, eo)], lengths, b)
    ref.check(o, ro, eo, "o")
    ref.check(hT, rS, eS, "hT")
    o2, none = ssd.ssd_linattn(**d, scale=dk ** -0.5, lengths=_lengths(lengths, dev), want_final=False)
    torch.cuda.synchronize()
    _cleared([(ro, eo)], lengths, b)
    assert none is None
    ref.check(o2, ro, eo, "o without a final state")


@pytest.mark.parametrize("case", LONG, ids=str)
def test_gradients_of_many_segments(case):
    dtype, b, L, G, H, dk, dv, decay, state, lengths = case
    dev = require_gpu()
    d = _grad_inputs(dtype, b, L, G, H, dk, dv, dev, decay, state, seed=40)
    if decay != "none":
        d["g"].mul_(0.125)                   # exact: slow decays, as above
    got = ssd.ssd_linattn_backward(**d, scale=dk ** -0.5, lengths=_lengths(lengths, dev))
    torch.cuda.synchronize()
    want = ref.backward(**d, scale=dk ** -0.5, lengths=lengths)
    _cleared(want[:4], lengths, b)
    for name, x, (r, e) in zip(GRADS, got, want):
        if x is not None:
            ref.check(x, r, e, name)


def test_outputs_that_are_not_wanted():
    """Without dg the walks for dq and dk are the prompt's own (scores rounded once; with dg in two
    parts): their values, not their bits; dv's walk is the same."""
    dev = require_gpu()
    d = _grad_inputs("bf16", 2, 400, 2, 4, 64, 64, dev, "token", True)
    every = ssd.ssd_linattn_backward(**d)
    some = ssd.ssd_linattn_backward(**d, want_dg=False, want_dh0=False)
    torch.cuda.synchronize()
    assert some[3] is None and some[4] is None and torch.equal(every[2], some[2])
    want = ref.backward(**d, scale=1.0)
    for name, x, y, (r, e) in zip(GRADS[:2], every, some, want):
        ref.check(x, r, e, name)
        ref.check(y, r, e, name + " without dg")


def _flat(outs):
    return [t for out in outs for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def _calls(d, h, freqs, at, lengths, **kw):
    """Rotation, prompt, its gradients and a token on the states `h` (updated in place)."""
    q, k = ssd.ssd_rotary(d["q"], d["k"], freqs, at, **kw)
    o, hT = ssd.ssd_linattn(q, k, d["v"], d["g"], d["h0"], scale=0.125, lengths=lengths, **kw)
    grads = ssd.ssd_linattn_backward(o, q, k, d["v"], d["g"], d["h0"], hT, scale=0.125, lengths=lengths, **kw)
    tq, tk, tv, tg = (t[:, 0] for t in (q, k, d["v"], d["g"]))
    return _flat([q, k, o, hT, grads, ssd.ssd_linattn_step(tq, tk, tv, h, tg, **kw), h])


def _setup(dev, seed, L=700):
    d = _grad_inputs("bf16", 2, L, 2, 4, 64, 72, dev, "token", True, seed=seed)
    return (d, d["h0"].clone(), ssd.rotary_frequencies(64, device=dev),
            torch.tensor([5, 1000], dtype=torch.int32, device=dev), _lengths([L, L // 3], dev))


def test_repeats_have_the_same_bits():
    dev = require_gpu()
    d, h, freqs, at, lengths = _setup(dev, 50)
    first = [t.clone() for t in _calls(d, h.clone(), freqs, at, lengths)]
    for _ in range(5):
        again = _calls(d, h.clone(), freqs, at, lengths)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_graph_replays():
    """Two graphs with memory of their own, replayed with refilled inputs and eager work between:
    the eager bits each time."""
    dev = require_gpu()
    d, h, freqs, at, lengths = _setup(dev, 51)
    states = [h.clone(), h.clone()]
    _calls(d, h.clone(), freqs, at, lengths)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = _calls(d, s, freqs, at, lengths)
        graphs.append((g, out))
    assert all(torch.equal(s, h) for s in states)               # capture ran nothing
    eager = h.clone()
    for rep in range(5):
        new = _grad_inputs("bf16", 2, 700, 2, 4, 64, 72, dev, "token", True, seed=60 + rep)
        for n in ("q", "k", "v", "g", "h0"):
            d[n].copy_(new[n])
        at.add_(700)
        want = _calls(d, eager, freqs, at, lengths)
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(x, y) for x, y in zip(want, out)), f"replay {rep}"


def test_step_plan_in_a_graph():
    dev = require_gpu()
    d = _inputs("bf16", 3, 6, 2, 4, 64, 48, dev, seed=52)
    rows = {n: torch.empty_like(d[n][:, 0].contiguous()) for n in "qkvg"}
    h, eager = d["h0"].clone(), d["h0"].clone()
    side = torch.cuda.Stream(dev)
    plan = ssd.LinattnStepPlan(rows["q"], rows["k"], rows["v"], h, rows["g"], stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        plan.run()
    torch.cuda.synchronize()
    assert torch.equal(h, d["h0"])
    for t in range(6):
        for n in "qkvg":
            rows[n].copy_(d[n][:, t])
        torch.cuda.synchronize()
        g.replay()
        o = ssd.ssd_linattn_step(*(d[n][:, t] for n in "qkv"), eager, d["g"][:, t])
        torch.cuda.synchronize()
        assert torch.equal(plan.y, o) and torch.equal(h, eager)


def test_two_streams_at_once():
    dev = require_gpu()
    cases = [_setup(dev, 53 + i, 6000) for i in range(2)]
    want = [_calls(d, h.clone(), *rest) for d, h, *rest in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in cases]
    for _ in range(3):
        got, own = [], [h.clone() for _, h, *_ in cases]
        torch.cuda.synchronize()
        for s, (d, _, *rest), h in zip(streams, cases, own):
            with torch.cuda.stream(s):
                got.append(_calls(d, h, *rest))
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(p, q))


def test_given_stream_gets_its_own_memory():
    """Outputs and workspaces of calls on a given stream are not what the current one freed."""
    dev = require_gpu()
    d, h, freqs, at, lengths = _setup(dev, 55, 2000)
    want = _calls(d, h.clone(), freqs, at, lengths)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        own = h.clone()
        freed = [torch.empty_like(t) for t in want for _ in range(2)]
        taken = {t.data_ptr() for t in freed}
        torch.cuda.synchronize()
        del freed
        got = _calls(d, own, freqs, at, lengths, stream=handle)
        assert not taken & {t.data_ptr() for t in got[:-1]}
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_given_workspaces():
    """Just as many bytes as the call asks for, whatever they held; fewer are refused."""
    dev = require_gpu()
    d = _grad_inputs("bf16", 2, 700, 2, 4, 64, 72, dev, "token", True, seed=56)
    do, dhT = d.pop("do"), d.pop("dhT")
    prob = ssd.linattn_problem(d["q"], d["v"])
    for need, call in (
            (ssd.ssd_linattn_workspace_bytes(prob), lambda **kw: ssd.ssd_linattn(**d, **kw)),
            (ssd.ssd_linattn_backward_workspace_bytes(prob),
             lambda **kw: ssd.ssd_linattn_backward(do, **d, dhT=dhT, **kw))):
        want = call()
        guarded = torch.full((need + 512,), 255, dtype=torch.uint8, device=dev)
        got = call(workspace=guarded[256:256 + need])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert (guarded[:256] == 255).all() and (guarded[256 + need:] == 255).all()
        with pytest.raises(Exception, match="(?i)workspace"):
            call(workspace=guarded[256:255 + need])
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=guarded.cpu())


def test_one_tensor_for_several_inputs():
    dev = require_gpu()
    d = _inputs("bf16", 1, 200, 2, 2, 64, 64, dev, seed=57)
    x = d["v"].contiguous()
    o, hT = ssd.ssd_linattn(x, x, x, d["g"], d["h0"])
    torch.cuda.synchronize()
    ro, eo, rS, eS = ref.forward(x, x, x, d["g"], d["h0"], 1.0)
    ref.check(o, ro, eo, "o")
    ref.check(hT, rS, eS, "hT")
    got = ssd.ssd_linattn_backward(x, x, x, x, d["g"], d["h0"], d["h0"])
    torch.cuda.synchronize()
    for name, y, (r, e) in zip(GRADS, got, ref.backward(x, x, x, x, d["g"], d["h0"], d["h0"], 1.0)):
        ref.check(y, r, e, name)


def test_given_outputs_between_other_memory():
    """Given outputs of odd sizes: nothing beside them is written."""
    dev = require_gpu()
    d = _grad_inputs("bf16", 2, 330, 1, 3, 72, 40, dev, "token", True, seed=58)
    dhT, do = d.pop("dhT"), d.pop("do")
    held = []

    def room(like):
        n = like.numel()
        whole = torch.full((n + 256,), 7.0, dtype=like.dtype, device=dev)
        held.append((whole, n))
        return whole[128:128 + n].view(like.shape)

    o, hT = ssd.ssd_linattn(**d)
    o2, hT2 = ssd.ssd_linattn(**d, o=room(o), hT=room(hT))
    grads = ssd.ssd_linattn_backward(do, **d, dhT=dhT)
    given = {n: room(t) for n, t in zip(GRADS, grads)}
    again = ssd.ssd_linattn_backward(do, **d, dhT=dhT, **given)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(hT, hT2)
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
    for whole, n in held:
        assert (whole[:128] == 7).all() and (whole[128 + n:] == 7).all()


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes behind the first one, and states past 2^32 bytes."""
    dev = require_gpu()
    pitch, L = 1 << 21, 1100
    wide = torch.empty(L * pitch, device=dev, dtype=torch.bfloat16)
    d = _grad_inputs("bf16", 1, L, 1, 2, 64, 64, dev, "token", True, seed=59)
    s, at = dict(d), 0
    for n in ("q", "k", "v", "g", "do"):
        w = d[n][0, 0].numel()
        s[n] = torch.as_strided(wide, (1, L, w), (L * pitch, pitch, 1), at).unflatten(2, d[n].shape[2:])
        s[n].copy_(d[n])
        at += 128
    freqs = ssd.rotary_frequencies(64, device=dev)
    outs = []
    for x in (d, s):
        fwd = {n: x[n] for n in ("q", "k", "v", "g", "h0")}
        outs.append(_flat([ssd.ssd_linattn(**fwd), ssd.ssd_linattn_backward(**x),
                           ssd.ssd_rotary(x["q"], x["k"], freqs)]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    del wide, s, outs
    b, H = 160, 128
    h = torch.ones(b, H, 256, 256, device=dev)
    q, k, v = (torch.ones(b, H, 256, device=dev) for _ in range(3))
    o = ssd.ssd_linattn_step(q, k, v, h)
    torch.cuda.synchronize()
    assert h.numel() * 4 > 1 << 32 and (o == 512).all() and (h == 2).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_block(dtype):
    """Rotated columns of a projection through a prompt, each head's norm and the gate, then tokens
    one by one from its state; against the 64-bit definitions chained.  Rotation, scores, state
    reads, outputs, gate and norm round to the type once each: six half steps of the 2-norm; fp32's
    sums are of fewer than 400 terms in each of four places."""
    dev = require_gpu()
    b, L, T, G, H, dk, dv = 2, 330, 3, 2, 4, 64, 48
    tol = 6 * 2.0 ** -8 if dtype == "bf16" else 4 * 400 * 2.0 ** -24
    gen = torch.Generator().manual_seed(70)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(TD[dtype])
    q, k, v, z = _columns(dev, rnd(b, L + T, G, dk), rnd(b, L + T, G, dk), rnd(b, L + T, H, dv),
                          rnd(b, L + T, H, dv))
    g = torch.nn.functional.logsigmoid(rnd(b, L + T, H).float() + 3).to(TD[dtype]).to(dev)
    w = (1 + 0.1 * torch.randn(H * dv, generator=gen)).to(dev)
    freqs, scale = ssd.rotary_frequencies(48, device=dev), dk ** -0.5
    first = torch.tensor([0, 70], dtype=torch.int32, device=dev)
    flat = lambda t: t.reshape(*t.shape[:-2], H * dv)
    norm = lambda o, t: ssd.ssd_norm(flat(o), w, flat(z[:, t]).contiguous(), ngroups=H, gate_after=True)

    qr, kr = ssd.ssd_rotary(q[:, :L].contiguous(), k[:, :L].contiguous(), freqs, first)
    o, h = ssd.ssd_linattn(qr, kr, v[:, :L].contiguous(), g[:, :L].contiguous(), scale=scale)
    outs = [norm(o, slice(0, L))]
    for t in range(L, L + T):
        qt, kt = ssd.ssd_rotary(q[:, t], k[:, t], freqs, first + t)
        o = ssd.ssd_linattn_step(qt, kt, v[:, t], h, g[:, t], scale=scale)
        outs.append(norm(o, t)[:, None])
    got = torch.cat(outs, 1).cpu().double()
    torch.cuda.synchronize()

    at = first[:, None].cpu() + torch.arange(L + T)
    qd, kd = (ref.rotary(x, freqs, at, False, False, 1.0)[0] for x in (q, k))
    od, _, hd, _ = ref.forward(qd, kd, v.double(), g.double(), None, scale)
    od = od * (od.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt() * w.cpu().double().view(H, dv)
    want = flat(od * torch.nn.functional.silu(z.cpu().double()))
    for x, r in ((got, want), (h.cpu().double(), hd)):
        assert (x - r).norm() <= tol * r.norm()


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_scales_of_any_sign(scale):
    dev = require_gpu()
    d = _grad_inputs("bf16", 1, 330, 1, 2, 64, 40, dev, "token", True, seed=71)
    grads = ssd.ssd_linattn_backward(**d, scale=scale)
    do, dhT = d.pop("do"), d.pop("dhT")
    o, hT = ssd.ssd_linattn(**d, scale=scale)
    torch.cuda.synchronize()
    if scale == 0:
        # what the last state's gradient gives is left
        last, bound = ref.last_state(*(ref.per_head(d[n], 2) for n in "kv"),
                                     ref.log_decays(d["g"], 1, 330, 2, None), dhT.cpu().double(),
                                     weight=0.0, back=True)
        assert (o == 0).all() and (grads[0] == 0).all()
        ref.check(grads[4], last, bound, "dh0")
    else:
        ro, eo, rS, eS = ref.forward(**d, scale=scale)
        ref.check(o, ro, eo, "o")
        ref.check(hT, rS, eS, "hT")
        for name, x, (r, e) in zip(GRADS, grads, ref.backward(do, **d, dhT=dhT, scale=scale)):
            ref.check(x, r, e, name)
