"""GPU tests of linear attention and rotary positions, beside those of test_gpu_linattn: refusals
through the binding, and the decays' gradient within the spread of its roundings."""
import pytest
import torch

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
