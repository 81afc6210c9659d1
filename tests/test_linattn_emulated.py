"""The kernels of linear attention and rotary positions, emulated on the CPU (kernel_emulator): no
access leaves an array, no LDS is read before it is written, the order in which waves reach
their accesses between two barriers changes no bit, and outputs lie within the bounds of
linattn_ref.  No GPU needed."""
import ctypes

import pytest
import torch

import kernel_emulator as emu
import linattn_ref as ref
import linattn_spread as spread
import state_space_sequence_cumsum_amd as ssd

TD = {"fp32": torch.float32, "bf16": torch.bfloat16}
BEHIND = 7.0        # what outputs hold before a call

CASES = [
    # dtype, b, L, G, H, dk, dv, decay, state, lengths
    ("bf16", 1, 1, 1, 1, 8, 8, "token", True, None),
    ("bf16", 1, 130, 1, 2, 64, 64, "token", True, None),
    ("fp32", 1, 130, 1, 2, 64, 64, "token", True, None),
    ("bf16", 1, 90, 1, 1, 128, 136, "token", True, None),
    ("fp32", 1, 90, 1, 1, 128, 40, "head", True, None),
    ("bf16", 1, 70, 1, 1, 256, 200, "token", True, None),
    ("fp32", 1, 70, 1, 2, 136, 136, "token", True, None),
    ("fp32", 1, 150, 1, 2, 256, 256, "token", True, None),
    ("bf16", 1, 150, 1, 1, 256, 256, "token", True, None),
    ("bf16", 3, 130, 1, 2, 40, 72, "token", False, [130, 0, 65]),
    ("bf16", 1, 321, 1, 1, 64, 64, "token", True, None),           # segments
    ("fp32", 2, 193, 1, 1, 40, 72, "token", True, [193, 70]),
]


def _inputs(dtype, b, L, G, H, dk, dv, decay, state, seed=3):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    td = TD[dtype]
    d = dict(q=rnd(b, L, G, dk).to(td), k=rnd(b, L, G, dk).to(td), v=rnd(b, L, H, dv).to(td), g=None)
    if decay == "head":
        d["g"] = -0.3 * torch.rand(H, generator=gen)
    elif decay == "token":
        d["g"] = (-0.3 * torch.rand(b, L, H, generator=gen) ** 3).to(td)
    d["h0"] = rnd(b, H, dv, dk) if state else None
    d["do"] = rnd(b, L, H, dv).to(td)
    d["dhT"] = rnd(b, H, dv, dk) if state else None
    return d


def _both_orders(fn, problem, inputs, outs, need=None):
    """The outputs [(shape, type)] of a call, after one with the waves in each order."""
    m, what = emu.Memory(), []
    try:
        for descending in (False, True):
            ptrs = [m.put(t) for t in inputs]
            at = [None if o is None else m.put(torch.full(*o[:1], BEHIND, dtype=o[1])) for o in outs]
            args = [ctypes.byref(problem), *ptrs, *at]
            if need is not None:
                args += [m.room(need) if need > 1 else None, need]
            what.append((emu.start(fn, (*args, None), descending), at, args))
        got = []
        for pid, at, _ in what:
            emu.finish(pid, fn)
            got.append([None if o is None else m.get(p, *o) for p, o in zip(at, outs)])
    finally:
        m.close()
    for x, y in zip(*got):
        if x is not None:
            assert torch.equal(x, y), "the waves' order changes an output"
    return got[0]


def _problem(dtype, b, L, G, H, dk, dv, decay, scale):
    return ssd.LinattnProblem(b, L, H, G, dk, dv, 0, 0, 0, 0, 0, scale,
                              {"none": 0, "head": 1, "token": 2}[decay], int(dtype == "bf16"))


def _unwritten(pairs, lengths):
    for r, e in pairs:
        for i, n in enumerate(lengths or []):
            r[i, n:], e[i, n:] = BEHIND, 0


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompts(case):
    dtype, b, L, G, H, dk, dv, decay, state, lengths = case
    d = _inputs(dtype, b, L, G, H, dk, dv, decay, state)
    do, dhT = d.pop("do"), d.pop("dhT")
    p = _problem(dtype, b, L, G, H, dk, dv, decay, dk ** -0.5)
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    o, hT = _both_orders("ssd_linattn", p, [*(d[n] for n in ("q", "k", "v", "g", "h0")), lt],
                         [((b, L, H, dv), TD[dtype]), ((b, H, dv, dk), torch.float32)],
                         emu.lib().ssd_linattn_workspace_bytes(ctypes.byref(p)))
    ro, eo, rS, eS = ref.forward(**d, scale=dk ** -0.5, lengths=lengths)
    _unwritten([(ro, eo)], lengths)
    ref.check(o, ro, eo, "o")
    ref.check(hT, rS, eS, "hT")


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients(case):
    dtype, b, L, G, H, dk, dv, decay, state, lengths = case
    d = _inputs(dtype, b, L, G, H, dk, dv, decay, state)
    p = _problem(dtype, b, L, G, H, dk, dv, decay, dk ** -0.5)
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    td = TD[dtype]
    outs = [((b, L, G, dk), td), ((b, L, G, dk), td), ((b, L, H, dv), td),
            ((b, L, H), td) if decay == "token" else None, ((b, H, dv, dk), torch.float32)]
    got = _both_orders("ssd_linattn_backward", p,
                       [*(d[n] for n in ("do", "q", "k", "v", "g", "h0", "dhT")), lt], outs,
                       emu.lib().ssd_linattn_backward_workspace_bytes(ctypes.byref(p)))
    want = ref.backward(**d, scale=dk ** -0.5, lengths=lengths)
    for name, x, (r, e) in zip(("dq", "dk", "dv", "dg", "dh0"), got, want):
        if x is None:
            continue
        if name != "dh0":
            _unwritten([(r, e)], lengths)
        ref.check(x, r, e, name)
    if decay == "token":
        parts, deviation = spread.decay_gradient(**d, scale=dk ** -0.5, lengths=lengths)
        value = sum(parts.values())
        _unwritten([(value, deviation)], lengths)
        spread.check(got[3], value, deviation, "dg within its spread")


@pytest.mark.parametrize("case", [
    ("bf16", 3, 2, 4, 8, 24, "token"), ("fp32", 1, 1, 2, 40, 72, "head"), ("bf16", 2, 1, 1, 128, 8, "token"),
    ("bf16", 1, 1, 1, 256, 200, "none")], ids=str)
def test_steps(case):
    dtype, b, G, H, dk, dv, decay = case
    d = _inputs(dtype, b, 1, G, H, dk, dv, decay, True)
    row = {n: t[:, 0] if t is not None and t.dim() > 1 else t for n, t in d.items() if n in "qkvg"}
    p = _problem(dtype, b, 1, G, H, dk, dv, decay, 0.5)
    # h is updated in place: one call
    m = emu.Memory()
    try:
        h, o = m.put(d["h0"]), m.put(torch.full((b, H, dv), BEHIND, dtype=TD[dtype]))
        args = (ctypes.byref(p), *(m.put(row[n]) for n in "qkvg"), h, o, None)
        emu.finish(emu.start("ssd_linattn_step", args, False), "ssd_linattn_step")
        o, h = m.get(o, (b, H, dv), TD[dtype]), m.get(h, (b, H, dv, dk), torch.float32)
    finally:
        m.close()
    ro, eo, rS, eS = ref.step(row["q"], row["k"], row["v"], row["g"], d["h0"], 0.5)
    ref.check(o, ro, eo, "o")
    ref.check(h, rS, eS, "h")


@pytest.mark.parametrize("case", [
    # dtype, b, L, heads, groups, width, rotated, interleaved
    ("bf16", 1, 9003, 2, 0, 32, 32, False),     # eight tokens a workgroup, three in the last one
    ("bf16", 3, 1367, 1, 1, 24, 20, True),      # two, one in the last one; single elements
    ("fp32", 2, 3, 2, 1, 100, 36, True),
    ("bf16", 1, 2, 1, 1, 4096, 4096, False),
], ids=str)
def test_rotations(case):
    dtype, b, L, hq, hk, w, rot, inter = case
    gen = torch.Generator().manual_seed(L)
    xs = [torch.randn(b, L, n, w, generator=gen).to(TD[dtype]) if n else None for n in (hq, hk)]
    first = torch.randint(0, 1 << 20, (b,), generator=gen, dtype=torch.int32)
    freqs = ssd.rotary_frequencies(rot)
    p = ssd.RotaryProblem(b, L, hq, hk, w, rot, 0, 0, 1.0, 1, int(inter), 0, int(dtype == "bf16"))
    ys = _both_orders("ssd_rotary", p, [*xs, freqs, first],
                      [None if x is None else (x.shape, x.dtype) for x in xs])
    at = first[:, None] + torch.arange(L, dtype=torch.int32)
    for x, y in zip(xs, ys):
        if x is not None:
            r, e = ref.rotary(x, freqs, at, inter, False, 1.0)
            ref.check(y, r, e, "rotated")
