"""GPU tests of the operators around the forward against 64-bit references (block_ref): the
short causal convolution, the selective scan and the block norms, alone and as a block runs
them.  Every bound is the reference's, element by element."""
import pytest
import torch

import block_ref as ref
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TD = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _slice_of(t, before, behind):
    """The same values as columns of a wider array (NaN around them)."""
    wide = torch.full((*t.shape[:-1], before + t.shape[-1] + behind), float("nan"),
                      device=t.device, dtype=t.dtype)
    wide[..., before:before + t.shape[-1]] = t
    return wide[..., before:before + t.shape[-1]]


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------
def _conv_inputs(dtype, b, L, c, k, dev, seed=0, bias=True, state=True):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    return (rnd(b, L, c).to(TD[dtype]).to(dev), (rnd(c, k) * 0.5).to(dev),
            rnd(c).to(dev) if bias else None,
            rnd(b, k - 1, c).to(TD[dtype]).to(dev) if state else None)


CONV_CASES = [
    # dtype, b, L, split, width, (columns before, behind), lengths, silu, bias, state
    ("fp32", 1, 1, [5], 4, (0, 0), None, True, True, True),
    ("bf16", 2, 2, [64], 4, (0, 0), None, True, True, True),
    ("bf16", 3, 3, [256, 64, 64], 4, (0, 0), None, True, True, False),
    ("bf16", 2, 33, [520, 16, 16], 4, (8, 24), None, True, True, True),
    ("bf16", 1, 257, [777], 3, (0, 0), None, True, False, True),
    ("fp32", 2, 65, [36, 4], 2, (4, 0), None, False, True, True),
    ("fp32", 4, 100, [1028], 4, (3, 2), [0, 1, 2, 100], True, True, True),
    ("bf16", 5, 70, [264, 8, 8], 4, (16, 8), [70, 0, 1, 2, 33], True, True, True),
    ("bf16", 4, 40, [24], 2, (0, 0), [0, 1, 40, 39], False, False, False),
    ("bf16", 3, 130, [2048, 33, 15], 3, (1, 2), [130, 128, 64], True, True, False),
    ("bf16", 2, 64, [2048, 256, 256], 4, (2048, 32), None, True, True, True),
    # wider arrays whose columns start off 16 bytes, and dense rows of an odd width
    ("bf16", 2, 19, [64, 8, 8], 4, (4, 4), None, True, True, True),
    ("fp32", 2, 19, [64, 8, 8], 4, (0, 2), None, True, True, True),
]


@pytest.mark.parametrize("case", CONV_CASES, ids=str)
def test_conv(case):
    dtype, b, L, split, k, cols, lengths, act, bias, state = case
    dev = require_gpu()
    c = sum(split)
    x, w, bv, s0 = _conv_inputs(dtype, b, L, c, k, dev, 1, bias, state)
    n = lengths or [L] * b
    for i, m in enumerate(n):          # what stands behind a sequence is not read
        x[i, m:] = float("nan")
    xs = _slice_of(x, *cols)
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
    ys = [torch.full((b, L, m), -7.0, device=dev, dtype=TD[dtype]) for m in split]
    out, final = ssd.ssd_conv(xs, w, bv, s0, silu=act, lengths=lt, split=split, y=ys)
    torch.cuda.synchronize()
    assert all(p is q for p, q in zip(out, ys))
    xr = x.clone()
    for i, m in enumerate(n):
        xr[i, m:] = 0
    y, ey, fin = ref.conv(xr, w, bv, s0, n, act)
    y_out = torch.cat(ys, -1)
    for i, m in enumerate(n):
        ref.check(y_out[i, :m], y[i, :m], ey[i, :m], f"y of sequence {i}")
        assert (y_out[i, m:] == -7.0).all(), "rows behind the sequence were written"
    assert torch.equal(final.cpu().double(), fin), "final state"


@pytest.mark.parametrize("dtype,c,k", [("bf16", 64, 4), ("fp32", 21, 3), ("bf16", 2560, 2)])
def test_conv_in_pieces(dtype, c, k):
    """A prompt in three calls, the state handed on in place (pieces shorter than the state
    among them), and the rest token by token: the same bits as one call."""
    dev = require_gpu()
    b, L = 2, 57
    x, w, bv, s0 = _conv_inputs(dtype, b, L, c, k, dev, 2)
    y_all, f_all = ssd.ssd_conv(x, w, bv, s0)
    state, parts = s0.clone(), []
    for lo, hi in ((0, 1), (1, 3), (3, 50)):
        y, f = ssd.ssd_conv(x[:, lo:hi].contiguous(), w, bv, state, final_state=state)
        assert f is state
        parts.append(y)
    for t in range(50, L):
        parts.append(ssd.ssd_conv_step(x[:, t].contiguous(), w, bv, state)[:, None])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(parts, 1), y_all) and torch.equal(state, f_all)


@pytest.mark.parametrize("dtype,c,split", [("bf16", 2560, [2048, 256, 256]), ("bf16", 1001, [1001]),
                                           ("fp32", 1024, [1024])])
def test_conv_token_tiles(dtype, c, split):
    """Every output is the same sum whichever tile its token falls into: a long prompt (tiles of
    32 tokens) gives the bits of its pieces (tiles of 8)."""
    dev = require_gpu()
    L = 16390
    x, w, bv, s0 = _conv_inputs(dtype, 1, L, c, 4, dev, 25)
    ys, f = ssd.ssd_conv(x, w, bv, s0, split=split)
    state, parts = s0.clone(), []
    for lo in range(0, L, 1500):
        y, _ = ssd.ssd_conv(x[:, lo:lo + 1500], w, bv, state, split=split, final_state=state)
        parts.append(y)
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        assert torch.equal(y, torch.cat([p[i] for p in parts], 1))
    assert torch.equal(f, state)


@pytest.mark.parametrize("dtype,b,split,k,cols,act,bias", [
    ("bf16", 1, [2048, 256, 256], 4, (2048, 32), True, True),
    ("bf16", 128, [520], 4, (0, 0), True, True),
    ("fp32", 3, [17, 5, 2], 3, (1, 0), False, False),
    ("bf16", 7, [33], 2, (0, 3), True, True),
    ("fp32", 2, [256, 64, 64], 4, (0, 4), True, True),
])
def test_conv_step(dtype, b, split, k, cols, act, bias):
    dev = require_gpu()
    c = sum(split)
    x, w, bv, state = _conv_inputs(dtype, b, 1, c, k, dev, 3, bias)
    y, ey, fin = ref.conv(x, w, bv, state, None, act)
    out = ssd.ssd_conv_step(_slice_of(x[:, 0], *cols), w, bv, state, silu=act, split=split)
    torch.cuda.synchronize()
    ref.check(torch.cat(out, -1), y[:, 0], ey[:, 0], "y")
    assert torch.equal(state.cpu().double(), fin)


@pytest.mark.parametrize("dtype,split,k,offset", [
    ("bf16", [9, 8, 31], 3, 1), ("bf16", [777], 4, 3), ("bf16", [8, 17], 2, 0), ("bf16", [64, 7], 4, 5),
    ("fp32", [5, 4, 7], 4, 1), ("fp32", [129], 2, 3), ("fp32", [64, 3], 3, 2)])
def test_conv_outputs_and_states_off_16_bytes(dtype, split, k, offset):
    """Outputs and states that start on any element, inside guarded buffers, the state in place:
    the values are those of arrays of their own, and nothing next to them is written."""
    dev = require_gpu()
    b, L, c, lengths = 3, 43, sum(split), [43, 1, 20]
    x, w, bv, s0 = _conv_inputs(dtype, b, L, c, k, dev, 31)
    y, ey, fin = ref.conv(x, w, bv, s0, lengths, True)

    def guarded(*shape):
        n = 1
        for m in shape:
            n *= m
        whole = torch.full((n + 24,), -7.0, device=dev, dtype=TD[dtype])
        return whole, whole[offset:offset + n].view(shape)

    def guards_hold(whole, view):
        n = view.numel()
        return bool((whole[:offset] == -7.0).all() and (whole[offset + n:] == -7.0).all())

    outs = [guarded(b, L, m) for m in split]
    whole_state, state = guarded(b, k - 1, c)
    state.copy_(s0)
    lt = torch.tensor(lengths, dtype=torch.int32, device=dev)
    ssd.ssd_conv(x, w, bv, state, lengths=lt, split=split, y=[v for _, v in outs],
                 final_state=state)
    torch.cuda.synchronize()
    got = torch.cat([v for _, v in outs], -1)
    for i, n in enumerate(lengths):
        ref.check(got[i, :n], y[i, :n], ey[i, :n], f"y of sequence {i}")
        assert (got[i, n:] == -7.0).all()
    assert torch.equal(state.cpu().double(), fin)
    assert all(guards_hold(*o) for o in outs) and guards_hold(whole_state, state)

    # the next token, from the same state
    x1 = x[:, 7]
    y, ey, fin = ref.conv(x1[:, None], w, bv, state.clone(), None, True)
    outs = [guarded(b, m) for m in split]
    ssd.ssd_conv_step(x1, w, bv, state, split=split, y=[v for _, v in outs])
    torch.cuda.synchronize()
    ref.check(torch.cat([v for _, v in outs], -1), y[:, 0], ey[:, 0], "y of a step")
    assert torch.equal(state.cpu().double(), fin)
    assert all(guards_hold(*o) for o in outs) and guards_hold(whole_state, state)


def test_conv_lengths_out_of_range_are_clamped():
    """Lengths are data on the device: below 0 counts as 0, above L as L."""
    dev = require_gpu()
    x, w, bv, s0 = _conv_inputs("bf16", 3, 20, 72, 4, dev, 4)
    y0 = [torch.full((3, 20, 72), 3.0, device=dev, dtype=torch.bfloat16) for _ in range(2)]
    outs = []
    for y, n in zip(y0, ([-5, 21, 1 << 30], [0, 20, 20])):
        outs.append(ssd.ssd_conv(x, w, bv, s0, y=y,
                                 lengths=torch.tensor(n, dtype=torch.int32, device=dev)))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---------------------------------------------------------------------------
# scan
# ---------------------------------------------------------------------------
def _scan_inputs(dtype, b, L, c, G, N, dev, seed=0, D=True, z=True, bias=True, h0=True, act=True,
                 spread=1.0):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    td = TD[dtype]
    dt = spread * rnd(b, L, c) - 3.0
    if not act:
        dt = torch.nn.functional.softplus(dt)
    d = dict(x=rnd(b, L, c).to(td), dt=dt.to(td),
             A=-torch.exp(torch.rand(c, N, generator=g) * 2.77),
             B=rnd(b, L, G, N).to(td), C=rnd(b, L, G, N).to(td),
             D=rnd(c) if D else None, z=(spread * rnd(b, L, c)).to(td) if z else None,
             dt_bias=0.3 * rnd(c) if bias else None, h0=rnd(b, c, N) if h0 else None)
    return {k: None if v is None else v.to(dev) for k, v in d.items()}


def _run_scan(d, act, **kw):
    return ssd.ssd_scan(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                        dt_bias=d["dt_bias"], h0=d["h0"], dt_softplus=act, **kw)


def _ref_scan(d, act, lengths=None):
    return ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"], d["h0"],
                    lengths, act)


SCAN_CASES = [
    # dtype, b, L, c, G, N, options
    ("fp32", 1, 1, 1, 1, 8, {}),
    ("bf16", 1, 1, 64, 1, 16, {}),
    ("fp32", 2, 7, 65, 1, 16, dict(z=False)),
    ("bf16", 2, 8, 100, 2, 16, dict(D=False)),
    ("bf16", 1, 9, 130, 1, 24, dict(h0=False)),
    ("fp32", 1, 33, 96, 3, 32, dict(bias=False)),
    ("bf16", 1, 64, 128, 2, 40, dict(act=False)),
    ("fp32", 2, 65, 40, 1, 48, dict(act=False, bias=False, D=False, z=False, h0=False)),
    ("bf16", 1, 127, 70, 1, 56, {}),
    ("fp32", 1, 129, 66, 2, 64, {}),
    ("bf16", 2, 300, 257, 1, 16, {}),
    ("fp32", 1, 700, 64, 1, 16, {}),
    ("bf16", 1, 1025, 192, 1, 16, dict(h0=False)),
    # every state size split into segments, with odd ends
    ("bf16", 2, 77, 70, 1, 8, {}),
    ("fp32", 1, 100, 130, 2, 24, {}),
    ("bf16", 3, 45, 33, 1, 48, {}),
    ("bf16", 1, 280, 70, 1, 24, {}),
    ("fp32", 1, 150, 40, 1, 40, {}),
    ("bf16", 1, 140, 66, 2, 48, {}),
    ("fp32", 1, 131, 33, 1, 56, {}),
    # enough channels for whole walks of a longer sequence
    ("bf16", 128, 37, 520, 1, 8, {}),
    ("fp32", 64, 33, 1024, 2, 16, {}),
    # one wave, a whole last wave, one token in the last wave of a short prompt
    ("fp32", 2, 16, 17, 1, 16, dict(h0=False)),
    ("bf16", 1, 256, 50, 2, 16, {}),
    ("bf16", 1, 241, 31, 1, 32, dict(z=False, D=False)),
    # short prompts of many channels: four lanes a channel, every state size
    ("bf16", 20, 50, 520, 1, 8, {}),
    ("fp32", 17, 33, 1030, 2, 16, {}),
    ("bf16", 17, 34, 1001, 1, 24, {}),
    ("bf16", 20, 49, 530, 1, 32, dict(h0=False)),
    ("fp32", 20, 33, 600, 1, 40, {}),
    ("bf16", 20, 40, 600, 1, 48, {}),
    ("bf16", 20, 40, 600, 1, 56, {}),
    ("fp32", 20, 35, 600, 1, 64, {}),
    # ... and of few: eight lanes
    ("bf16", 1, 33, 66, 1, 32, {}),
    ("fp32", 1, 20, 30, 1, 40, {}),
    ("bf16", 2, 128, 24, 1, 64, {}),
    # step sizes from e^-23 to 17: the far ends of the softplus
    ("fp32", 1, 200, 64, 1, 16, dict(spread=8.0)),
    ("bf16", 2, 90, 64, 1, 8, dict(spread=8.0)),
]


@pytest.mark.parametrize("case", SCAN_CASES, ids=str)
def test_scan(case):
    dtype, b, L, c, G, N, opt = case
    dev = require_gpu()
    act = opt.get("act", True)
    d = _scan_inputs(dtype, b, L, c, G, N, dev, 5, **opt)
    y = torch.full((b, L, c), float("nan"), device=dev, dtype=TD[dtype])
    hT = torch.full((b, c, N), float("nan"), device=dev)
    _run_scan(d, act, y=y, hT=hT)
    torch.cuda.synchronize()
    ry, ey, rh, eh = _ref_scan(d, act)
    ref.check(y, ry, ey, "y")
    ref.check(hT, rh, eh, "hT")


@pytest.mark.parametrize("dtype,L,c,G,N,lengths", [
    ("bf16", 40, 70, 1, 16, [0, 1, 40, 39]),
    ("fp32", 300, 130, 2, 8, [300, 0, 150, 64]),
    ("bf16", 1100, 64, 1, 32, [3, 1100, 512, 513]),
])
def test_scan_ragged(dtype, L, c, G, N, lengths):
    """A padded batch: rows behind a sequence hold NaN, their outputs stay as they were, and
    the final state is the one after the sequence's own last token (h0 for none)."""
    dev = require_gpu()
    b = len(lengths)
    d = _scan_inputs(dtype, b, L, c, G, N, dev, 6)
    clean = {k: None if v is None else v.clone() for k, v in d.items()}
    for i, m in enumerate(lengths):
        for k in ("x", "dt", "B", "C", "z"):
            d[k][i, m:] = float("nan")
            clean[k][i, m:] = 0
    y = torch.full((b, L, c), -7.0, device=dev, dtype=TD[dtype])
    _, hT = _run_scan(d, True, y=y, lengths=torch.tensor(lengths, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    ry, ey, rh, eh = _ref_scan(clean, True, lengths)
    for i, m in enumerate(lengths):
        ref.check(y[i, :m], ry[i, :m], ey[i, :m], f"y of sequence {i}")
        assert (y[i, m:] == -7.0).all()
        if m == 0:
            assert torch.equal(hT[i], d["h0"][i])
    ref.check(hT, rh, eh, "hT")


@pytest.mark.parametrize("dtype,b,c,G,N", [
    ("bf16", 1024, 9, 1, 8), ("fp32", 512, 66, 1, 16), ("bf16", 512, 6, 2, 24),
    ("fp32", 1030, 5, 1, 32), ("bf16", 1024, 4, 1, 40), ("fp32", 1024, 3, 1, 48),
    ("bf16", 512, 4, 2, 56), ("fp32", 1024, 2, 1, 64), ("bf16", 1024, 3, 1, 64)])
def test_scan_ragged_batch_of_whole_walks(dtype, b, c, G, N):
    """A wave for each of 1024 sequences or more, with every length from none to all tokens."""
    dev = require_gpu()
    L = 70
    lengths = [(i * 37) % (L + 1) for i in range(b)]
    d = _scan_inputs(dtype, b, L, c, G, N, dev, 41)
    past = torch.arange(L)[None, :] >= torch.tensor(lengths)[:, None]
    past = past.to(dev)
    clean = {k: None if v is None else v.clone() for k, v in d.items()}
    for k in ("x", "dt", "B", "C", "z"):
        d[k][past] = float("nan")
        clean[k][past] = 0
    y = torch.full((b, L, c), -7.0, device=dev, dtype=TD[dtype])
    _, hT = _run_scan(d, True, y=y, lengths=torch.tensor(lengths, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    ry, ey, rh, eh = _ref_scan(clean, True, lengths)
    assert (y[past] == -7.0).all(), "rows behind a sequence were written"
    live = ~past.cpu()
    ref.check(y.cpu()[live], ry[live], ey[live], "y")
    ref.check(hT, rh, eh, "hT")
    empty = [i for i, n in enumerate(lengths) if n == 0]
    assert torch.equal(hT[empty], d["h0"][empty])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_column_slices(dtype):
    """Inputs that are columns of wider arrays give the bits of dense ones."""
    dev = require_gpu()
    d = _scan_inputs(dtype, 2, 75, 132, 2, 16, dev, 7)
    y0, h0 = _run_scan(d, True)
    s = dict(d)
    s["x"], s["dt"], s["z"] = (_slice_of(d[k], *cols) for k, cols in
                               (("x", (1, 2)), ("dt", (0, 5)), ("z", (132, 0))))
    for k, cols in (("B", (48, 32)), ("C", (2, 0))):
        s[k] = _slice_of(d[k].flatten(2), *cols).unflatten(2, (2, 16))
    y1, h1 = _run_scan(s, True)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(h0, h1)


def test_scan_state_in_place_and_continued():
    """hT in h0's own buffer, and a prompt in two calls and then steps: the whole prompt's."""
    dev = require_gpu()
    for L, cut in ((25, 3), (90, 37), (1500, 1200)):
        d = _scan_inputs("fp32", 2, L, 80, 1, 16, dev, 8)
        ry, ey, rh, eh = _ref_scan(d, True)
        h = d["h0"].clone()
        part = dict(d, h0=h, **{k: d[k][:, :cut].contiguous() for k in ("x", "dt", "B", "C", "z")})
        y1, hT = _run_scan(part, True, hT=h)
        assert hT is h
        part = dict(d, h0=h, **{k: d[k][:, cut:L - 5].contiguous() for k in ("x", "dt", "B", "C", "z")})
        y2, _ = _run_scan(part, True, hT=h)
        ys = [y1, y2]
        for t in range(L - 5, L):
            ys.append(ssd.ssd_scan_step(
                *(d[k][:, t].contiguous() if k != "A" else d[k] for k in ("x", "dt", "A", "B", "C")),
                h, D=d["D"], z=d["z"][:, t].contiguous(), dt_bias=d["dt_bias"],
                dt_softplus=True)[:, None])
        torch.cuda.synchronize()
        ref.check(torch.cat(ys, 1), ry, ey, "y")
        ref.check(h, rh, eh, "h")


def test_scan_zero_step_keeps_state_bitwise():
    dev = require_gpu()
    for L in (5, 100, 2000):
        d = _scan_inputs("fp32", 1, L, 64, 1, 16, dev, 9, act=False, bias=False)
        d["dt"].zero_()
        _, hT = _run_scan(d, False)
        torch.cuda.synchronize()
        assert torch.equal(hT, d["h0"])


@pytest.mark.parametrize("L", [200, 400])
def test_scan_zero_state_under_growing_rates(L):
    """Positive rates: a segment's decay overflows, but a state that is still zero stays zero,
    as it does token by token."""
    dev = require_gpu()
    d = _scan_inputs("fp32", 1, L, 64, 1, 16, dev, 22, h0=False, act=False, bias=False)
    d["A"] = -d["A"]
    d["dt"].fill_(1.0)
    d["x"][:, :-2] = 0
    y, hT = _run_scan(d, False)
    torch.cuda.synchronize()
    ry, ey, rh, eh = _ref_scan(d, False)
    ref.check(y, ry, ey, "y")
    ref.check(hT, rh, eh, "hT")


def test_scan_many_segments():
    """A long prompt of few channels: more segments than a chain workgroup holds at once."""
    dev = require_gpu()
    d = _scan_inputs("fp32", 1, 20011, 9, 1, 8, dev, 27, spread=0.5)
    y, hT = _run_scan(d, True)
    torch.cuda.synchronize()
    ry, ey, rh, eh = _ref_scan(d, True)
    ref.check(y, ry, ey, "y")
    ref.check(hT, rh, eh, "hT")


def test_scan_without_final_state():
    dev = require_gpu()
    for L in (1, 20, 200, 1300):
        d = _scan_inputs("bf16", 2, L, 130, 1, 16, dev, 26)
        y0, hT = _run_scan(d, True)
        y1, none = _run_scan(d, True, want_final=False)
        torch.cuda.synchronize()
        assert hT is not None and none is None and torch.equal(y0, y1)


def test_scan_repeats_bitwise():
    """No atomics: the same call gives the same bits."""
    dev = require_gpu()
    d = _scan_inputs("bf16", 1, 3000, 256, 1, 16, dev, 10)
    y0, h0 = _run_scan(d, True)
    for _ in range(3):
        y1, h1 = _run_scan(d, True)
        torch.cuda.synchronize()
        assert torch.equal(y0, y1) and torch.equal(h0, h1)


@pytest.mark.parametrize("dtype,b,c,G,N,opt", [
    ("bf16", 1, 2048, 1, 16, {}),
    ("fp32", 3, 65, 1, 8, dict(D=False)),
    ("bf16", 128, 96, 2, 24, dict(z=False)),
    ("bf16", 2, 130, 1, 40, dict(bias=False)),
    ("fp32", 2, 63, 3, 56, dict(act=False)),
    ("bf16", 5, 200, 2, 64, {}),
    ("fp32", 2, 100, 1, 32, {}),
    ("bf16", 2, 100, 1, 48, {}),
])
def test_scan_step(dtype, b, c, G, N, opt):
    dev = require_gpu()
    act = opt.get("act", True)
    d = _scan_inputs(dtype, b, 1, c, G, N, dev, 11, **opt)
    ry, ey, rh, eh = _ref_scan(d, act)
    h = d["h0"].clone()
    t = {k: None if d[k] is None else d[k][:, 0] for k in ("x", "dt", "B", "C", "z")}
    y = ssd.ssd_scan_step(_slice_of(t["x"], 1, 2), t["dt"], d["A"], t["B"], t["C"], h, D=d["D"],
                          z=t["z"], dt_bias=d["dt_bias"], dt_softplus=act)
    torch.cuda.synchronize()
    ref.check(y, ry[:, 0], ey[:, 0], "y")
    ref.check(h, rh, eh, "h")


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
NORM_CASES = [
    # dtype, rows, channels, groups, gate, residual type, columns around x and z
    ("fp32", 1, 1, 1, "none", None, (0, 0)),
    ("bf16", 1, 8, 1, "first", None, (0, 0)),
    ("bf16", 3, 64, 4, "after", None, (0, 0)),
    ("fp32", 5, 63, 3, "first", "fp32", (1, 2)),
    ("bf16", 2, 255, 1, "none", "fp32", (0, 0)),
    ("bf16", 7, 1024, 1, "none", "bf16", (0, 0)),
    ("bf16", 4, 2048, 1, "first", None, (0, 2592)),
    ("bf16", 4, 2048, 2, "after", "fp32", (2048, 0)),
    ("fp32", 3, 4096, 1, "first", "fp32", (0, 0)),
    ("bf16", 2, 8192, 1, "first", "bf16", (8, 8)),
    ("bf16", 2, 8200, 1, "none", "fp32", (0, 0)),
    ("fp32", 2, 20000, 1, "after", None, (0, 0)),
    ("bf16", 300, 96, 1, "first", "fp32", (0, 4)),
    ("bf16", 2, 20001, 1, "first", "bf16", (0, 0)),
    ("fp32", 9, 516, 1, "none", None, (0, 0)),
    # teams that walk over several rows: waves, workgroups, parts of a wave, three groups
    ("bf16", 9001, 1024, 1, "first", None, (0, 0)),
    ("bf16", 2100, 4096, 1, "none", "bf16", (0, 0)),
    ("fp32", 70003, 32, 1, "after", None, (0, 0)),
    ("bf16", 4001, 1032, 3, "first", "fp32", (0, 8)),
    # single elements in a wave, and in a workgroup
    ("bf16", 5, 999, 1, "after", "bf16", (0, 0)),
    ("fp32", 3, 1501, 1, "first", "fp32", (0, 0)),
    ("bf16", 4, 2049, 1, "none", "fp32", (0, 0)),
    ("bf16", 2300, 4095, 1, "first", None, (1, 0)),
]


def _norm_inputs(dtype, rows, c, gate, residual, dev, seed=0):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    x, z = rnd(rows, c).to(TD[dtype]).to(dev), (2 * rnd(rows, c)).to(TD[dtype]).to(dev)
    r = (4 * rnd(rows, c)).to(dev)
    return (x, (1 + 0.2 * rnd(c)).to(dev), None if gate == "none" else z,
            None if residual is None else r.to(TD[residual]))


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_norm(case):
    dtype, rows, c, G, gate, residual, cols = case
    dev = require_gpu()
    x, w, z, r = _norm_inputs(dtype, rows, c, gate, residual, dev, 12)
    kw = dict(ngroups=G, eps=1e-5, scale=0.3, gate_after=gate == "after")
    out = ssd.ssd_norm(_slice_of(x, *cols), w, None if z is None else _slice_of(z, *cols), r, **kw)
    torch.cuda.synchronize()
    y, ey, v, ev = ref.norm(x, w, z, r, **kw)
    if r is None:
        return ref.check(out, y, ey, "y")
    ref.check(out[0], y, ey, "y")
    ref.check(out[1], v, ev, "residual")


@pytest.mark.parametrize("c", [2048, 511])
def test_norm_residual_in_place_and_zero_rows(c):
    """The residual stream updated in its own buffer; a row of zeros gives zeros."""
    dev = require_gpu()
    x, w, _, r = _norm_inputs("bf16", 6, c, "none", "fp32", dev, 13)
    x[2], r[2] = 0, 0
    y0, v0 = ssd.ssd_norm(x, w, residual=r, scale=0.5)
    rin = r.clone()
    y1, v1 = ssd.ssd_norm(x, w, residual=rin, residual_out=rin, scale=0.5)
    y2, v2 = ssd.ssd_norm(x, w, residual=r, scale=0.5, want_residual=False)
    torch.cuda.synchronize()
    assert v1 is rin and v2 is None
    assert torch.equal(y0, y1) and torch.equal(v0, v1) and torch.equal(y0, y2)
    assert (y0[2] == 0).all() and (v0[2] == 0).all()


@pytest.mark.parametrize("dtype,c", [("fp32", 64), ("bf16", 2049), ("fp32", 20000)])
def test_norm_smallest_eps(dtype, c):
    """The smallest eps: rows of zeros, and of elements whose squares vanish next to it or not."""
    dev = require_gpu()
    x = torch.zeros(4, c, dtype=TD[dtype])
    x[1], x[2, ::2], x[3, 1] = 1e-18, -1e-22, 3.0
    w = torch.linspace(-2, 2, c)
    y, ey, _, _ = ref.norm(x, w, eps=2.0 ** -126)
    out = ssd.ssd_norm(x.to(dev), w.to(dev), eps=2.0 ** -126)
    torch.cuda.synchronize()
    assert (out[0] == 0).all()
    # (the squares of row 2 are subnormal, 1e-44: as many digits of y as they have are not asked for)
    ref.check(out[[0, 1, 3]], y[[0, 1, 3]], ey[[0, 1, 3]], "y")
    assert torch.isfinite(out).all()


def test_norm_takes_leading_dimensions():
    dev = require_gpu()
    x, w, z, _ = _norm_inputs("bf16", 12, 128, "first", None, dev, 14)
    y = ssd.ssd_norm(x, w, z)
    wide = _slice_of(x, 0, 128)
    y3 = ssd.ssd_norm(wide.unflatten(0, (3, 4)), w, z.view(3, 4, 128))
    torch.cuda.synchronize()
    assert y3.shape == (3, 4, 128) and torch.equal(y3.view(12, 128), y)


# ---------------------------------------------------------------------------
# far offsets, streams, graphs, plans
# ---------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """Rows that lie more than 2^32 bytes behind the first: 1030 tokens at a pitch of 2^21
    elements."""
    dev = require_gpu()
    pitch, L, c = 1 << 21, 1030, 72
    wide = torch.empty(L * pitch, device=dev, dtype=torch.bfloat16)
    col = lambda off, w: torch.as_strided(wide, (1, L, w), (L * pitch, pitch, 1), off)
    x, w, bv, _ = _conv_inputs("bf16", 1, L, c, 4, dev, 15)
    xs = col(0, c)
    xs.copy_(x)
    y0, f0 = ssd.ssd_conv(x, w, bv)
    y1, f1 = ssd.ssd_conv(xs, w, bv)
    assert torch.equal(y0, y1) and torch.equal(f0, f1)
    d = _scan_inputs("bf16", 1, L, c, 1, 16, dev, 16)
    s = dict(d)
    for i, k in enumerate(("x", "dt", "z", "B", "C")):
        v = d[k].flatten(2)
        s[k] = col(128 * (i + 1), v.shape[2])
        s[k].copy_(v)
    s["B"], s["C"] = s["B"].unflatten(2, (1, 16)), s["C"].unflatten(2, (1, 16))
    y0, h0 = _run_scan(d, True)
    y1, h1 = _run_scan(s, True)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    wn = torch.ones(c, device=dev)
    assert torch.equal(ssd.ssd_norm(d["x"], wn, d["z"]), ssd.ssd_norm(s["x"], wn, s["z"]))


def _block_calls(d, conv, norm, state, h):
    """conv -> scan -> gated norm, as a block runs them."""
    u, cs = ssd.ssd_conv(conv[0], conv[1], conv[2], state)
    y, hT = ssd.ssd_scan(u, d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["dt_bias"], h0=h,
                         dt_softplus=True)
    return ssd.ssd_norm(y, norm[0], d["z"]), cs, hT


def test_side_stream_and_graph_replays():
    """The three operators on a side stream and captured into a graph (allocating its own
    outputs and workspace from the graph's pool): every replay, with eager work and refilled
    inputs between, gives the eager bits."""
    dev = require_gpu()
    b, L, c = 2, 700, 128
    d = _scan_inputs("bf16", b, L, c, 1, 16, dev, 17)
    conv = _conv_inputs("bf16", b, L, c, 4, dev, 18)
    norm = (torch.ones(c, device=dev),)
    want = _block_calls(d, conv, norm, conv[3], d["h0"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    with torch.cuda.stream(side):
        got = _block_calls(d, conv, norm, conv[3], d["h0"])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = _block_calls(d, conv, norm, conv[3], d["h0"])
        graphs.append((g, out))
    for rep in range(4):
        conv[0].copy_(torch.randn(b, L, c, generator=_gen(40 + rep)))
        d["dt"].copy_(torch.randn(b, L, c, generator=_gen(50 + rep)) - 3)
        want = _block_calls(d, conv, norm, conv[3], d["h0"])
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(want, out)), f"replay {rep}"


def test_given_stream_gets_its_own_memory():
    """Outputs and workspaces of a call on a given stream come from that stream's memory, not
    from what the current stream has just freed and may still be using."""
    dev = require_gpu()
    side = torch.cuda.Stream(dev)
    b, L, c = 1, 4096, 256
    d = _scan_inputs("bf16", b, L, c, 1, 16, dev, 23)
    conv = _conv_inputs("bf16", b, L, c, 4, dev, 24)
    w = torch.ones(c, device=dev)
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        freed = [torch.empty(b, L, c, device=dev, dtype=torch.bfloat16) for _ in range(8)]
        freed += [torch.empty(b, c, 16, device=dev) for _ in range(4)]
        taken = {t.data_ptr() for t in freed}
        del freed
        u, cs = ssd.ssd_conv(conv[0], conv[1], stream=handle)
        y, hT = _run_scan(d, True, stream=handle)
        o = ssd.ssd_norm(d["x"], w, stream=handle)
        assert not taken & {t.data_ptr() for t in (u, y, hT, o)}
        torch.cuda.synchronize()
        want = ssd.ssd_conv(conv[0], conv[1])[0], *_run_scan(d, True), ssd.ssd_norm(d["x"], w)
        assert all(torch.equal(p, q) for p, q in zip((u, y, hT, o), want))


def test_two_streams_at_once():
    """Calls in flight on two streams share nothing: the bits of calls in turn."""
    dev = require_gpu()
    cases = [(_scan_inputs("bf16", 1, 6000, 256, 1, 16, dev, 30 + i),
              _conv_inputs("bf16", 1, 6000, 256, 4, dev, 32 + i)) for i in range(2)]
    norm = (torch.ones(256, device=dev),)
    want = [_block_calls(d, conv, norm, conv[3], d["h0"]) for d, conv in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in cases]
    for _ in range(3):
        got = []
        for s, (d, conv) in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(_block_calls(d, conv, norm, conv[3], d["h0"]))
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_refusals():
    """What a call cannot take raises, with nothing launched: the next call's outputs are right."""
    dev = require_gpu()
    bf, f32 = torch.bfloat16, torch.float32
    z = lambda *s, dtype=bf: torch.zeros(*s, device=dev, dtype=dtype)
    x, w = z(2, 5, 64), z(64, 4, dtype=f32)
    for kw in (dict(weight=z(64, 4)), dict(weight=z(63, 4, dtype=f32)), dict(bias=z(64)),
               dict(state=z(2, 2, 64)), dict(split=[32, 33]), dict(split=[64, 0]),
               dict(split=[16] * 4), dict(lengths=torch.zeros(2, device=dev, dtype=torch.int64)),
               dict(lengths=torch.zeros(2, dtype=torch.int32)), dict(y=z(2, 5, 32)),
               dict(y=z(2, 64, 5).mT), dict(x=x.expand(3, 2, 5, 64)[0][:1].expand(2, 5, 64)),
               dict(x=z(2, 5, 128)[:, :, ::2]), dict(x=z(2, 9, 64)[:, :5]), dict(x=x[0])):
        with pytest.raises(ValueError):
            ssd.ssd_conv(**{**dict(x=x, weight=w), **kw})
    for k in (1, 5):
        with pytest.raises(ssd.SsdError) as err:
            ssd.ssd_conv(x, z(64, k, dtype=f32))
        assert err.value.status == 3
    with pytest.raises(ssd.SsdError) as err:      # weights that start off 16 bytes
        ssd.ssd_conv(x, z(64 * 4 + 1, dtype=f32)[1:].view(64, 4))
    assert err.value.status == 6

    d = dict(x=x, dt=x, A=z(64, 16, dtype=f32), B=z(2, 5, 1, 16), C=z(2, 5, 1, 16))
    for kw in (dict(A=z(64, 16)), dict(A=z(64, 8, dtype=f32)), dict(C=z(2, 5, 2, 16)), dict(dt=z(2, 5, 63)),
               dict(h0=z(2, 64, 16)), dict(D=z(64)), dict(z=x.float()), dict(dt_bias=z(63, dtype=f32)),
               dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)), dict(x=x[:, 0])):
        with pytest.raises(ValueError):
            ssd.ssd_scan(**{**d, **kw})
    with pytest.raises(ssd.SsdError) as err:
        ssd.ssd_scan(**{**d, "A": z(64, 12, dtype=f32), "B": z(2, 5, 1, 12), "C": z(2, 5, 1, 12)})
    assert err.value.status == 3
    with pytest.raises(ssd.SsdError) as err:      # bf16 rows of B that start off 4 bytes
        ssd.ssd_scan(**{**d, "B": z(2, 5, 18)[:, :, 1:17].unflatten(2, (1, 16))})
    assert err.value.status == 6
    long = {k: (v if k == "A" else v.repeat_interleave(200, 1)) for k, v in d.items()}
    with pytest.raises(ssd.SsdError) as err:
        ssd.ssd_scan(**long, workspace=z(16, dtype=torch.uint8))
    assert err.value.status == 4
    with pytest.raises(ValueError):
        ssd.ssd_scan_step(x[:, 0], x[:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], None)
    with pytest.raises(ValueError):
        ssd.ssd_conv_step(x[:, 0], w, None, None)

    for kw in (dict(weight=z(64)), dict(z=z(2, 5, 63)), dict(residual=z(2, 5, 64, dtype=torch.float16)),
               dict(residual_out=z(2, 5, 64)), dict(y=x.float())):
        with pytest.raises(ValueError):
            ssd.ssd_norm(**{**dict(x=x, weight=z(64, dtype=f32)), **kw})
    for kw in (dict(eps=0.0), dict(scale=float("inf")), dict(eps=float("nan"))):
        with pytest.raises(ssd.SsdError) as err:
            ssd.ssd_norm(x, z(64, dtype=f32), **kw)
        assert err.value.status == 3
    with pytest.raises(ssd.SsdError) as err:
        ssd.ssd_norm(x, z(64, dtype=f32), ngroups=3)
    assert err.value.status == 2
    y = ssd.ssd_norm(torch.ones(1, 64, device=dev), torch.ones(64, device=dev))
    assert abs(float(y[0, 0]) - 1) < 1e-4


@pytest.mark.parametrize("workspace", [1 << 20, [0], "4096", b"0"], ids=repr)
def test_workspace_that_is_no_tensor_is_refused(workspace):
    dev = require_gpu()
    d = _scan_inputs("bf16", 1, 1000, 64, 1, 16, dev, 77)
    with pytest.raises(ValueError, match="workspace"):
        _run_scan(d, True, workspace=workspace)


def test_step_plans_and_graph():
    """ConvStepPlan and ScanStepPlan captured into one decode graph, inputs refilled between
    the replays: the states and outputs of the eager steps, bit for bit."""
    dev = require_gpu()
    b, T, c = 3, 6, 192
    d = _scan_inputs("bf16", b, T, c, 1, 16, dev, 19)
    conv = _conv_inputs("bf16", b, T, c, 4, dev, 20)
    x = torch.empty(b, c, device=dev, dtype=torch.bfloat16)
    dt, z = torch.empty_like(x), torch.empty_like(x)
    B = torch.empty(b, 1, 16, device=dev, dtype=torch.bfloat16)
    C = torch.empty_like(B)
    cs, h = conv[3].clone(), d["h0"].clone()
    side = torch.cuda.Stream(dev)
    cp = ssd.ConvStepPlan(x, conv[1], conv[2], cs, stream=side)
    sp = ssd.ScanStepPlan(cp.y, dt, d["A"], B, C, h, D=d["D"], z=z, dt_bias=d["dt_bias"],
                          dt_softplus=True, stream=side)
    cs2, h2 = conv[3].clone(), d["h0"].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cp.run()
        sp.run()
    torch.cuda.synchronize()
    assert torch.equal(cs, conv[3]) and torch.equal(h, d["h0"])      # capture ran nothing
    for t in range(T):
        x.copy_(conv[0][:, t]); dt.copy_(d["dt"][:, t]); z.copy_(d["z"][:, t])
        B.copy_(d["B"][:, t]); C.copy_(d["C"][:, t])
        torch.cuda.synchronize()
        g.replay()
        u = ssd.ssd_conv_step(conv[0][:, t], conv[1], conv[2], cs2)
        y = ssd.ssd_scan_step(u, d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], h2, D=d["D"],
                              z=d["z"][:, t], dt_bias=d["dt_bias"], dt_softplus=True)
        torch.cuda.synchronize()
        assert torch.equal(cp.y, u) and torch.equal(sp.y, y)
        assert torch.equal(cs, cs2) and torch.equal(h, h2)


# ---------------------------------------------------------------------------
# as a block runs them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_block_around_the_forward(dtype):
    """Convolution of the projection's x, B and C columns, the SSD forward on its split
    outputs, the gated norm and the next block's residual norm; then two tokens through the
    decode forms.  Against the 64-bit definitions chained, to the forward's own bar."""
    dev = require_gpu()
    b, L, T, H, P, N = 2, 200, 2, 4, 64, 64
    c = H * P
    td, tol = TD[dtype], {"bf16": 2e-2, "fp32": 1e-4}[dtype]
    g = _gen(21)
    rnd = lambda *s: torch.randn(*s, generator=g)
    proj = rnd(b, L + T, 2 * c + 2 * N + H).to(td).to(dev)         # z, x, B, C, dt
    w, bias = (0.5 * rnd(c + 2 * N, 4)).to(dev), (0.1 * rnd(c + 2 * N)).to(dev)
    A, D = -torch.exp(rnd(H)).to(dev), torch.rand(H, generator=g).to(dev)
    dt = torch.nn.functional.softplus(proj[..., -H:].float() - 4).to(td)
    nw, nw2 = (1 + 0.1 * rnd(c)).to(dev), (1 + 0.1 * rnd(c)).to(dev)
    res = rnd(b, L + T, c).to(dev)
    z, xbc = proj[..., :c], proj[..., c:2 * c + 2 * N]

    (x, B, C), cs = ssd.ssd_conv(xbc[:, :L].contiguous(), w, bias, split=[c, N, N])
    y, h = ssd.ssd_forward(x.view(b, L, H, P), dt[:, :L].contiguous(), A, B.view(b, L, 1, N),
                           C.view(b, L, 1, N), D, chunk=64)
    y = ssd.ssd_norm(y.view(b, L, c), nw, z[:, :L].contiguous())
    out, stream = ssd.ssd_norm(y, nw2, residual=res[:, :L].contiguous(), scale=0.5)
    outs, streams = [out], [stream]
    for t in range(L, L + T):
        x, B, C = ssd.ssd_conv_step(xbc[:, t], w, bias, cs, split=[c, N, N])
        y = ssd.ssd_step(x.view(b, H, P), dt[:, t].contiguous(), A, B.view(b, 1, N),
                         C.view(b, 1, N), D, h)
        y = ssd.ssd_norm(y.view(b, c), nw, z[:, t])
        o, s = ssd.ssd_norm(y, nw2, residual=res[:, t].contiguous(), scale=0.5)
        outs.append(o[:, None])
        streams.append(s[:, None])
    torch.cuda.synchronize()

    v, _, fin = ref.conv(xbc.contiguous(), w, bias, None, None, True)
    rep = lambda t: t.cpu().double().repeat_interleave(P, -1)
    yr, _, hr, _ = ref.scan(v[..., :c], rep(dt), rep(A)[:, None].expand(c, N), v[..., None, c:c + N],
                            v[..., None, c + N:], rep(D))
    yr, _, _, _ = ref.norm(yr.flatten(0, 1), nw, z.reshape(-1, c))
    yo, _, so, _ = ref.norm(yr, nw2, None, res.view(-1, c), scale=0.5)
    for got, want, what in ((torch.cat(outs, 1).view(-1, c), yo, "out"),
                            (torch.cat(streams, 1).view(-1, c), so, "residual stream"),
                            (h.view(b, c, N), hr, "state"), (cs, fin, "conv state")):
        err = ((ref.d64(got) - want).abs().max() / want.abs().max()).item()
        print(f"  {what}: {err:.2e}", flush=True)
        assert err <= tol, (what, err)


# ---------------------------------------------------------------------------
# shared memory: what is refused, and what the single-token forms and the norm allow
# ---------------------------------------------------------------------------
def test_outputs_in_inputs_are_refused():
    """Before any launch: the inputs keep their values."""
    dev = require_gpu()
    x, w, bv, s0 = _conv_inputs("bf16", 2, 40, 64, 4, dev, 71)
    d = _scan_inputs("bf16", 2, 40, 64, 1, 16, dev, 72)
    kept = [t.clone() for t in (x, s0, d["x"], d["z"], d["h0"])]
    long = {k: v.repeat_interleave(30, 1) if k in ("x", "dt", "B", "C", "z") else v for k, v in d.items()}
    ws = torch.empty(1 << 24, device=dev, dtype=torch.uint8)
    calls = [
        lambda: ssd.ssd_conv(x, w, bv, s0, y=x),
        lambda: ssd.ssd_conv(x[:1], w, bv, s0[:1], y=x.view(-1)[64:64 * 41].view(1, 40, 64)),
        lambda: ssd.ssd_conv(x, w, bv, s0, split=[32, 32], y=[torch.empty(2, 40, 32, device=dev, dtype=x.dtype)] * 2),
        lambda: ssd.ssd_conv(x, w, bv, x.view(-1)[:2 * 3 * 64].view(2, 3, 64), final_state=x.view(-1)[64:7 * 64].view(2, 3, 64)),
        lambda: _run_scan(d, True, y=d["x"]),
        lambda: _run_scan(d, True, y=d["z"]),
        lambda: _run_scan(long, True, workspace=ws, hT=ws[1 << 10:].view(torch.float32)[:2 * 64 * 16].view(2, 64, 16)),
        lambda: ssd.ssd_norm(d["x"], torch.ones(64, device=dev), residual=d["z"], y=d["x"], residual_out=d["x"]),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ssd.SsdError) as err:
            call()
        assert err.value.status == 9, i
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(kept, (x, s0, d["x"], d["z"], d["h0"])))


def test_outputs_between_the_rows_of_wide_inputs():
    """A dense output in the columns next to a wider array's rows shares nothing with them."""
    dev = require_gpu()
    x, w, bv, s0 = _conv_inputs("bf16", 1, 3, 8, 4, dev, 73)
    want, f0 = ssd.ssd_conv(x, w, bv, s0)
    wide = torch.zeros(3, 64, device=dev, dtype=torch.bfloat16)
    wide[:, 16:24] = x[0]
    y = wide[0, 32:56].view(1, 3, 8)              # 24 elements between the rows of tokens 0 and 1
    got, f1 = ssd.ssd_conv(wide[None, :, 16:24], w, bv, s0, y=y)
    torch.cuda.synchronize()
    assert got is y and torch.equal(got, want) and torch.equal(f0, f1)
    assert torch.equal(wide[:, 16:24], x[0])


@pytest.mark.parametrize("dtype,c", [("bf16", 96), ("fp32", 33), ("bf16", 20001)])
def test_steps_and_norms_in_place(dtype, c):
    """A step's and a norm's output in the buffer of x (or of the gate, the step sizes, the
    residual stream): the bits of an output of its own."""
    dev = require_gpu()
    x, w, z, r = _norm_inputs(dtype, 37, c, "first", dtype, dev, 74)
    for kw in (dict(z=z), dict(z=z, residual=r, scale=0.5), dict(z=z, gate_after=True)):
        want = ssd.ssd_norm(x, w, **kw)
        for k in ("x", "z") + (("residual",) if "residual" in kw else ()):
            t = {"x": x, **kw}
            t[k] = t[k].clone()
            got = ssd.ssd_norm(weight=w, y=t[k], **t)
            torch.cuda.synchronize()
            both = zip(got, want) if "residual" in kw else ((got, want),)
            assert all(torch.equal(p, q) for p, q in both), (kw.keys(), k)
    if c > 10000:
        return
    x, w, bv, s0 = _conv_inputs(dtype, 5, 1, c, 4, dev, 75)
    s1, a = s0.clone(), x[:, 0].clone()
    want = ssd.ssd_conv_step(x[:, 0].clone(), w, bv, s0)
    assert ssd.ssd_conv_step(a, w, bv, s1, y=a) is a
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(s0, s1)
    d = _scan_inputs(dtype, 5, 1, c, 1, 16, dev, 76)
    t = {k: d[k][:, 0].contiguous() for k in ("x", "dt", "B", "C", "z")}
    h0 = d["h0"].clone()
    want = ssd.ssd_scan_step(t["x"], t["dt"], d["A"], t["B"], t["C"], h0, z=t["z"], dt_softplus=True)
    for k in ("x", "dt", "z"):
        u, h1 = {**t, k: t[k].clone()}, d["h0"].clone()
        got = ssd.ssd_scan_step(u["x"], u["dt"], d["A"], u["B"], u["C"], h1, z=u["z"],
                                dt_softplus=True, y=u[k])
        torch.cuda.synchronize()
        assert got is u[k] and torch.equal(got, want) and torch.equal(h0, h1), k
