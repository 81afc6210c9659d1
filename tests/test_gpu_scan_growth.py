"""GPU tests of scans whose states grow or shrink by more than fp32's range holds as one factor:
exp of a run's summed steps overflows (or is zero) although every state along the way is an
ordinary number.  Against the 64-bit recurrence, element by element."""
import pytest
import torch

import block_ref as ref
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

# b, L, groups, channels a group, dstate; roundings of a run's summed steps: the tokens of a
# segment (or of a wave in the one-launch form), and the 16 segments of a chain's run
SHAPES = [
    (2, 200, 1, 64, 16, 16),          # one launch, 13 waves of eight lanes a channel
    (1, 128, 1, 70, 64, 16),          # one launch, 64 states
    (16, 200, 10, 2, 8, 16),          # one launch, four lanes a channel
    (1, 2000, 1, 64, 8, 8 + 16),      # segments of 8 tokens
    (8, 5003, 16, 2, 8, 64 + 16),     # segments of 64 tokens, 1024 chains
]


def _growth(shape, tokens, total, size, sign):
    """One state per channel and n whose logarithm moves by about `total` over the first `tokens`
    tokens and then stays: steps and rates of `sign` (so that sign * sign has total's sign)."""
    b, L, G, cg, N, run = shape
    g = torch.Generator().manual_seed(tokens)
    c = G * cg
    A = sign * (0.9 + 0.1 * torch.rand(c, N, generator=g))
    dt = torch.zeros(b, L, c)
    dt[:, :tokens] = sign * total / tokens
    magnitude = size * 10.0 ** (2 * torch.rand(b, c, N, generator=g) - 1)
    h0 = magnitude * (1 - 2 * torch.randint(0, 2, (b, c, N), generator=g))
    d = dict(x=torch.zeros(b, L, c), dt=dt, A=A, B=torch.randn(b, L, G, N, generator=g),
             C=torch.randn(b, L, G, N, generator=g), h0=h0)
    return d, run


def _compare(d, run, dev):
    y, hT = ssd.ssd_scan(*(d[k].to(dev) for k in ("x", "dt", "A", "B", "C")), h0=d["h0"].to(dev))
    torch.cuda.synchronize()
    ry, ey, rh, eh = ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], h0=d["h0"], run=run)
    assert not torch.isinf(eh).any()
    ref.check(hT, rh, eh, "hT")
    ref.check(y, ry, ey, "y")


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("tokens", [8, 16, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_small_states_grow(shape, tokens, sign):
    """States of 1e-31 to 1e-29 that grow by e^99 to e^110."""
    dev = require_gpu()
    _compare(*_growth(shape, tokens, 110.0, 1e-30, sign), dev)


@pytest.mark.parametrize("tokens", [8, 16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_subnormal_states_grow(shape, tokens):
    """States of 1e-41 to 1e-39, below the smallest normal number, that grow by e^135 to e^150
    (by e^8 or more in the first token, so that no product is itself subnormal)."""
    dev = require_gpu()
    _compare(*_growth(shape, tokens, 150.0, 1e-40, 1.0), dev)


@pytest.mark.parametrize("tokens", [8, 16, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_large_states_shrink(shape, tokens):
    """States of 1e29 to 1e31 that shrink by e^-126 to e^-140, more than the smallest number."""
    dev = require_gpu()
    d, run = _growth(shape, tokens, 140.0, 1e30, 1.0)
    d["A"] = -d["A"]
    _compare(d, run, dev)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_growth_between_inputs(shape):
    """Growth by e^85 and decay back in turn, every 24 tokens, with small inputs all along."""
    dev = require_gpu()
    b, L, G, cg, N, run = shape
    d, _ = _growth(shape, 1, 0.0, 1e-30, 1.0)
    at = torch.arange(L) % 48
    d["dt"] = torch.where(at < 24, 3.5, -3.5)[None, :, None].expand(b, L, G * cg).contiguous()
    d["x"] = 1e-30 * torch.randn(b, L, G * cg, generator=torch.Generator().manual_seed(3))
    _compare(d, run, dev)
