"""GPU tests of linear attention and rotary positions, beside those of test_gpu_linattn: refusals
through the binding, the decays' gradient within the spread of its roundings, rotations whose
last workgroup has fewer tokens."""
import pytest
import torch

import linattn_ref as ref
import linattn_spread as spread
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu
from linattn_cases import ONE_CHUNK, SPREAD, inputs, one_chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
def test_gradients_of_too_many_heads_are_refused(given):
    """Rows of all heads' dq and dk past the limit: refused, with every output as it was."""
    dev = require_gpu()
    new = lambda *s: torch.ones(s, device=dev, dtype=torch.bfloat16)
    q, v, g = new(1, 64, 1, 256), new(1, 64, 16392, 8), -new(1, 64, 16392)
    outs = {}
    if given:
        outs = dict(dq=3 * new(*q.shape), dk=3 * new(*q.shape), dv=3 * new(*v.shape), dg=3 * new(*g.shape),
                    workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev))
    with pytest.raises(ssd.SsdError) as e:
        ssd.ssd_linattn_backward(v, q, q, v, g, **outs)
    torch.cuda.synchronize()
    assert e.value.status == 3
    assert all((outs[n] == 3).all() for n in outs if n != "workspace")


@pytest.mark.parametrize("rate", [0.3, 0.03])
@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_the_decays_gradient_within_its_spread(case, rate):
    dtype, b, L, G, H, dk, dv, state, lengths = case
    dev = require_gpu()
    d = inputs(case, dev, seed=60, rate=rate)
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)
    dg = ssd.ssd_linattn_backward(**d, scale=dk ** -0.5, lengths=lt)[3]
    torch.cuda.synchronize()
    parts, deviation = spread.decay_gradient(**d, scale=dk ** -0.5, lengths=lengths)
    spread.check(dg, sum(parts.values()), deviation, "dg")


@pytest.mark.parametrize("part", ONE_CHUNK)
def test_one_chunks_decays_gradient_is_rounded_once(part):
    """Scores and states that the decays' gradient is made of go in as two parts: of 2048 elements the
    error is that of one rounding, 1 +- 0.02 (1.4 with either in one part)."""
    dev = require_gpu()
    d = one_chunk(part, dev, 61)
    dg = ssd.ssd_linattn_backward(**d, scale=0.125)[3]
    torch.cuda.synchronize()
    parts, _ = spread.decay_gradient(**d, scale=0.125)
    assert spread.one_rounding(dg, sum(parts.values())) < 1.1


@pytest.mark.parametrize("case", [
    # dtype, b, L, heads, groups, width, rotated, interleaved, positions: tokens of a workgroup, of the last one
    ("bf16", 1, 4099, 2, 1, 128, 128, False, "first"),      # 4, 3
    ("bf16", 1, 9003, 2, 0, 64, 32, True, "first"),         # 8, 3
    ("fp32", 3, 4777, 3, 1, 100, 36, True, "each"),         # 8, 3
    ("bf16", 7, 2341, 2, 1, 24, 20, False, "each"),         # 8, 3 (single elements)
    ("fp32", 1, 32783, 1, 1, 32, 32, False, "start"),       # 16, 15
], ids=str)
def test_rotations_whose_last_workgroup_is_not_full(case):
    dtype, b, L, hq, hk, w, rot, inter, mode = case
    dev = require_gpu()
    gen = torch.Generator().manual_seed(L)
    td = torch.float32 if dtype == "fp32" else torch.bfloat16
    xs = [torch.randn(b, L, n, w, generator=gen).to(td).to(dev) for n in (hq, hk) if n]
    t = torch.arange(L, dtype=torch.int32)
    given = {"start": None, "first": torch.randint(0, 1 << 20, (b,), generator=gen, dtype=torch.int32),
             "each": torch.randint(0, 1 << 20, (b, L), generator=gen, dtype=torch.int32)}[mode]
    at = t.expand(b, L) if given is None else given[:, None] + t if mode == "first" else given
    freqs = ssd.rotary_frequencies(rot, device=dev)
    # outputs with the same bytes behind them afterwards
    wide = [torch.full((x.numel() + 4096,), 7.0, device=dev, dtype=td) for x in xs]
    outs = [t[:x.numel()].view(x.shape) for t, x in zip(wide, xs)]
    ssd.ssd_rotary(xs[0], xs[1] if hk else None, freqs, None if given is None else given.to(dev),
                   interleaved=inter, q_out=outs[0], k_out=outs[1] if hk else None)
    torch.cuda.synchronize()
    for x, y, whole in zip(xs, outs, wide):
        r, e = ref.rotary(x, freqs, at, inter, False, 1.0)
        ref.check(y, r, e, "rotated")
        assert (whole[x.numel():] == 7).all()
