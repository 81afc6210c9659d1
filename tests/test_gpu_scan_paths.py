"""GPU tests of the scan's paths by what selects them: segments of every rule of the split, chains
over many segments, the one-launch form with many waves.  Against the 64-bit recurrence, element
by element, with the roundings of a run's summed steps counted as they are made.

Groups of few channels give many waves (each owns channels of one group) for little work."""
import pytest
import torch

import block_ref as ref
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu
from test_gpu_block import TD, _run_scan, _scan_inputs

pytestmark = pytest.mark.gpu


def _segments(dtype, b, L, G, cg, N):
    """How many segments the library splits these sequences into, from its workspace: per
    segment N states and a sum of steps for each of 64 lanes of a wave (1: no workspace)."""
    p = ssd.ScanProblem(b, L, G * cg, G, N, 0, 0, 0, 0, 0, 1,
                        ssd.SSD_BF16 if TD[dtype] == torch.bfloat16 else ssd.SSD_F32)
    n = ssd.ssd_scan_workspace_bytes(p)
    return 1 if n == 1 else n // (b * (N + 1) * G * -(-cg // 64) * 64 * 4)


def _check(d, lengths, run, dev, act=True):
    b, L, c = d["x"].shape
    n = lengths or [L] * b
    past = (torch.arange(L)[None, :] >= torch.tensor(n)[:, None]).to(dev)
    clean = {k: None if v is None else v.clone() for k, v in d.items()}
    for k in ("x", "dt", "B", "C", "z"):
        if d[k] is not None:
            d[k][past] = float("nan")
            clean[k][past] = 0
    y = torch.full_like(d["x"], -7.0)
    lt = None if lengths is None else torch.tensor(n, dtype=torch.int32, device=dev)
    _, hT = _run_scan(d, act, y=y, lengths=lt)
    torch.cuda.synchronize()
    ry, ey, rh, eh = ref.scan(*(clean[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")),
                              n, act, run=run)
    assert (y[past] == -7.0).all(), "rows behind a sequence were written"
    live = ~past.cpu()
    ref.check(y.cpu()[live], ry[live], ey[live], "y")
    ref.check(hT, rh, eh, "hT")
    if 0 in n and d["h0"] is not None:
        assert torch.equal(hT[n.index(0)], d["h0"][n.index(0)])


# dtype, b, L, groups, channels a group, dstate; tokens of a segment that the split takes, segments
SPLITS = [
    ("bf16", 2, 2900, 12, 2, 16, 24, 121),      # up to 4096 waves of fewer than 32 tokens
    ("fp32", 4, 8200, 4, 2, 64, 32, 257),       # 32 tokens, 1024 chains, three rounds of a chain
    ("bf16", 4, 9001, 8, 3, 16, 40, 226),       # up to 8192 waves of 32 to 64 tokens, 512 chains
    ("fp32", 8, 5003, 16, 2, 8, 64, 79),        # 64 tokens, 1024 chains
    ("bf16", 1, 16390, 32, 1, 16, 64, 257),     # 64 tokens of one sequence, 512 chains
    ("bf16", 3, 3500, 20, 70, 24, 56, 63),      # two waves a group, the second nearly empty
    ("fp32", 3, 3600, 100, 1, 8, 72, 50),       # up to 16384 waves of more than 64 tokens
    ("bf16", 100, 1200, 10, 1, 8, 80, 15),      # ... 1000 waves, 8000 chains
    ("fp32", 31, 700, 33, 1, 32, 64, 11),       # 1023 waves: the most that are split
]


@pytest.mark.parametrize("ragged", [False, True], ids=["dense", "ragged"])
@pytest.mark.parametrize("case", SPLITS, ids=str)
def test_split_scans(case, ragged):
    """Dense, and with lengths at and around segment ends."""
    dtype, b, L, G, cg, N, seg, segments = case
    dev = require_gpu()
    assert _segments(dtype, b, L, G, cg, N) == segments == -(-L // seg)
    d = _scan_inputs(dtype, b, L, G * cg, G, N, dev, 81)
    lengths = None
    if ragged:
        ends = [L, 0, seg, seg + 1, 2 * seg - 1, 1, 16 * seg, 16 * seg + 1, L - 1, 17 * seg - 1, 3]
        lengths = [min(ends[i % len(ends)] + i // len(ends), L) for i in range(b)]
        if b == 1:
            lengths = [128 * seg + 1]          # one segment, of one token, behind a chain's round
    _check(d, lengths, seg + 16, dev)


# dtype, b, L, groups, channels a group, dstate, lanes of a channel
SHORTS = [
    # five or more waves, four lanes a channel: 2049 to 4096 waves of 16 tokens, every state size
    ("bf16", 16, 200, 10, 2, 8, 4), ("fp32", 4, 200, 1, 700, 16, 4), ("bf16", 13, 256, 10, 2, 24, 4),
    ("fp32", 13, 256, 10, 1, 32, 4), ("bf16", 8, 256, 1, 512, 32, 4), ("fp32", 26, 128, 10, 2, 40, 4),
    ("bf16", 60, 65, 7, 3, 48, 4), ("fp32", 40, 97, 9, 1, 56, 4), ("bf16", 8, 128, 1, 700, 64, 4),
    # eight lanes
    ("bf16", 6, 256, 1, 70, 16, 8), ("fp32", 7, 241, 2, 9, 32, 8), ("bf16", 6, 128, 3, 10, 64, 8),
    ("fp32", 6, 100, 2, 20, 40, 8),
]


@pytest.mark.parametrize("ragged", [False, True], ids=["dense", "ragged"])
@pytest.mark.parametrize("case", SHORTS, ids=str)
def test_one_launch_with_many_waves(case, ragged):
    """Dense, and with lengths at and around the ends of a wave's 16 tokens, whole waves of the
    workgroup behind them."""
    dtype, b, L, G, cg, N, lanes = case
    dev = require_gpu()
    assert _segments(dtype, b, L, G, cg, N) == 1
    waves = -(-L // 16)
    four = waves * b * G * -(-cg // 16)
    assert waves > 4 and (four <= 2048 if lanes == 8 else 2048 < four <= 4096)
    d = _scan_inputs(dtype, b, L, G * cg, G, N, dev, 82)
    lengths = None
    if ragged:
        ends = [L, 0, 1, 16, 17, 129, 31, L - 1, 64, 65, 80]
        lengths = [min(ends[i % len(ends)] + i // len(ends), L) for i in range(b)]
    _check(d, lengths, 16, dev)


def test_long_prompt_of_the_listed_size():
    """16384 tokens of 2048 channels, 16 states, gate and softplus (segments of 64 tokens), on
    every 64th channel and the ends of a wave."""
    dev = require_gpu()
    L, c, N = 16384, 2048, 16
    assert _segments("bf16", 1, L, 1, c, N) == 256
    d = _scan_inputs("bf16", 1, L, c, 1, N, dev, 83)
    y, hT = _run_scan(d, True)
    torch.cuda.synchronize()
    at = sorted({*range(0, c, 64), *range(63, c, 256), 1, c - 2})
    few = {k: v[..., at].contiguous() if k in ("x", "dt", "z", "D", "dt_bias") else v for k, v in d.items()}
    few["A"], few["h0"] = d["A"][at], d["h0"][:, at]
    ry, ey, rh, eh = ref.scan(*(few[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")),
                              None, True, run=64 + 16)
    ref.check(y[..., at], ry, ey, "y")
    ref.check(hT[:, at], rh, eh, "hT")
