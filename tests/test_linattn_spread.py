"""The reference of the decays' gradient that adds up variances (linattn_spread): its parts are the
gradient, a gradient with the roundings that it counts passes, and one with a part missing or
wrong does not.  No GPU needed."""
import pytest
import torch

import linattn_ref as ref
import linattn_spread as spread
from linattn_cases import ONE_CHUNK, SPREAD, inputs, one_chunk


@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_a_wrong_part_is_seen(case):
    dtype, b, L, G, H, dk, dv, state, lengths = case
    d = inputs(case, "cpu")
    parts, deviation = spread.decay_gradient(**d, scale=dk ** -0.5, lengths=lengths)
    value = sum(parts.values())
    whole = ref.backward(**d, scale=dk ** -0.5, lengths=lengths)[3][0]
    for i, n in enumerate(lengths or []):
        whole[i, n:] = 0
    assert torch.allclose(value, whole, rtol=1e-9, atol=1e-9 * whole.abs().max().item())

    td = d["q"].dtype
    assert not spread.misses(value.to(td), value, deviation, td).any()
    share = lambda x: spread.misses(x.to(td), value, deviation, td).double().sum().item()
    for name, part in parts.items():
        # a part that is there at all: missing in most of its elements, seen in nearly all of them
        there = (part.abs() > 0.05 * value.abs().clamp_min(value.norm() / value.numel() ** 0.5)).double().sum().item()
        if there > 0:
            assert share(value - part) >= 0.9 * there, name
            assert share(value - 0.25 * part) >= 0.5 * there, name + " in part"
        # a token's part at the next one (inside a chunk, parts of cross are alike)
        if there > 0 and name != "cross":
            assert share(value - part + part.roll(1, 1)) >= 0.25 * there, name + " moved"
    assert share(1.02 * value) >= 0.25 * value.count_nonzero()


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_counted_roundings_pass(seed):
    """States handed over in bf16: the part that crosses chunks errs by what the deviation says."""
    case = ("bf16", 1, 300, 2, 2, 64, 64, True, None)
    d = inputs(case, "cpu", seed)
    scale = 0.125
    parts, deviation = spread.decay_gradient(**d, scale=scale)
    value = sum(parts.values())
    # the same states again, rounded
    g = ref.log_decays(d["g"], 1, 300, 2, None)
    q, k, v, do = (ref.per_head(d[n], 2) for n in ("q", "k", "v", "do"))
    p = ref.Pairs(g)
    S = ref.states(k, v, d["h0"].double(), p)
    dS = ref.states(q, do * scale, d["dhT"].double(), ref.Pairs(g, True))
    rounded = value.clone()
    for c in range(p.chunks):
        s = slice(c * 64, min((c + 1) * 64, 300))
        before = p.G[..., s.start - 1:s.start] if c else 0.0
        e = ((S[:, :, c].bfloat16().double() - S[:, :, c]) * dS[:, :, c]).sum((2, 3))[..., None]
        rounded[:, s] += (e * (p.G[..., s.stop - 1:s.stop] - before).exp()).transpose(1, 2)
    assert not spread.misses(rounded.bfloat16(), value, deviation, torch.bfloat16).any()
    # the deviation is that of the roundings, not several times theirs
    off = (rounded - value).norm() / deviation.norm()
    assert 0.2 < off < 2.0


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("part", ONE_CHUNK)
def test_an_operand_rounded_once_is_seen(part, seed):
    """One chunk's gradient rounded once errs by one rounding (2048 elements: 1 +- 0.02 standard
    deviations); with scores or states in one bf16 part before, by more than 1.2."""
    d = one_chunk(part, "cpu", seed)
    parts, _ = spread.decay_gradient(**d, scale=0.125)
    value = sum(parts.values())
    assert 0.9 < spread.one_rounding(value.bfloat16(), value) < 1.1
    g = ref.log_decays(d["g"], 8, 64, 4, None)
    q, k, v, do = (ref.per_head(d[n], 4) for n in ("q", "k", "v", "do"))
    p, once = ref.Pairs(g), lambda x: x.bfloat16().double()
    upto = torch.ones(64, 64, dtype=torch.float64).tril()
    if part == "inside":
        # only the pairs' own scores of reads: the same in both walks
        m = torch.matmul(q, k.transpose(2, 3)) * once(torch.matmul(do, v.transpose(2, 3)) * p.D * 0.125)
        wrong = (torch.matmul(m.transpose(2, 3), upto) * (1 - upto)).sum(2)
        wrong = wrong.transpose(1, 2) - parts["inside"]
    elif part == "read":
        x = (torch.matmul(q, once(d["h0"]).transpose(2, 3)) * do).sum(3) * p.G.exp() * 0.125
        wrong = torch.matmul(x, upto).transpose(1, 2) - parts["read"]
    else:
        x = (torch.matmul(k, once(d["dhT"]).transpose(2, 3)) * v).sum(3) * (p.G[..., -1:] - p.G).exp()
        wrong = torch.matmul(x, 1 - upto).transpose(1, 2) - parts["written"]
    assert spread.one_rounding((value + wrong).bfloat16(), value) > 1.2
