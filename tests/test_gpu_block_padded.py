"""GPU tests of padded batches (`lengths`) as a block runs them: the convolution's outputs go on
into ssd_forward, which has no lengths, and the outputs that a call allocates itself hold zeros
behind each sequence."""
import pytest
import torch

import block_ref as ref
import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu
from test_gpu_block import _conv_inputs, _run_scan, _scan_inputs

pytestmark = pytest.mark.gpu

TD = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _fill_free_memory(dev, dtype, *counts):
    """NaN in the memory that the next allocations of these element counts are taken from."""
    held = [torch.full((n,), float("nan"), device=dev, dtype=dtype) for n in counts for _ in range(6)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("dtype,split", [("bf16", [72]), ("fp32", [33, 5]), ("bf16", [256, 64, 64]),
                                         ("bf16", [7, 9, 11])])
def test_conv_allocates_zeros_behind_sequences(dtype, split):
    dev = require_gpu()
    lengths, L, c = [50, 0, 1, 49, 17], 50, sum(split)
    x, w, bias, s0 = _conv_inputs(dtype, 5, L, c, 4, dev, 61)
    lt = torch.tensor(lengths, dtype=torch.int32, device=dev)
    given = [torch.zeros(5, L, m, device=dev, dtype=TD[dtype]) for m in split]
    _, f0 = ssd.ssd_conv(x, w, bias, s0, lengths=lt, split=split, y=given)
    _fill_free_memory(dev, TD[dtype], *(5 * L * m for m in split), 5 * L * c)
    ys, f1 = ssd.ssd_conv(x, w, bias, s0, lengths=lt, split=split)
    torch.cuda.synchronize()
    for y, z in zip(ys, given):
        assert y.is_contiguous() and y.data_ptr() % 16 == 0 and torch.equal(y, z)
    assert torch.equal(f0, f1)


@pytest.mark.parametrize("L", [40, 200, 900])
def test_scan_allocates_zeros_behind_sequences(L):
    dev = require_gpu()
    lengths = [L, 0, 1, L // 2, L - 1]
    d = _scan_inputs("bf16", 5, L, 70, 1, 16, dev, 62)
    lt = torch.tensor(lengths, dtype=torch.int32, device=dev)
    given = torch.zeros(5, L, 70, device=dev, dtype=torch.bfloat16)
    _, h0 = _run_scan(d, True, lengths=lt, y=given)
    _fill_free_memory(dev, torch.bfloat16, 5 * L * 70)
    y, h1 = _run_scan(d, True, lengths=lt)
    torch.cuda.synchronize()
    assert torch.equal(y, given) and torch.equal(h0, h1)


def test_zeros_on_a_given_stream():
    """The clearing runs on the call's own stream, before its kernels."""
    dev = require_gpu()
    L, split, lengths = 4000, [256, 32], [4000, 7]
    x, w, bias, s0 = _conv_inputs("bf16", 2, L, 288, 4, dev, 66)
    lt = torch.tensor(lengths, dtype=torch.int32, device=dev)
    want = [torch.zeros(2, L, m, device=dev, dtype=x.dtype) for m in split]
    ssd.ssd_conv(x, w, bias, s0, lengths=lt, split=split, y=want)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        for _ in range(5):
            with torch.cuda.stream(side):
                _fill_free_memory(dev, x.dtype, 2 * L * 288 + 256)
            ys, _ = ssd.ssd_conv(x, w, bias, s0, lengths=lt, split=split, stream=handle)
            side.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(ys, want))


def test_padded_calls_in_a_graph():
    """Captured, every replay clears the rows behind the sequences of that replay's lengths."""
    dev = require_gpu()
    L, split = 90, [64, 16]
    x, w, bias, s0 = _conv_inputs("bf16", 3, L, 80, 4, dev, 63)
    d = _scan_inputs("bf16", 3, L, 64, 1, 16, dev, 64)
    lt = torch.tensor([L, 5, 0], dtype=torch.int32, device=dev)

    def calls():
        ys, f = ssd.ssd_conv(x, w, bias, s0, lengths=lt, split=split)
        y, h = _run_scan(dict(d, x=ys[0]), True, lengths=lt)
        return (*ys, f, y, h)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = calls()
    for n in ([L, 5, 0], [1, L, 44], [0, 0, L], [3, 3, 3]):
        lt.copy_(torch.tensor(n, dtype=torch.int32))
        want = calls()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, out)), n
        for y in (want[0], want[1], want[3]):
            for i, m in enumerate(n):
                assert (y[i, m:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padded_batch_through_the_forward(dtype):
    """Convolution with lengths, the SSD forward on its outputs with step sizes of zero behind
    each sequence, the gated norm: valid tokens and final states are those of each sequence by
    itself, to the forward's own bar."""
    dev = require_gpu()
    lengths, L, H, P, N = [200, 77, 1, 130], 200, 4, 64, 64
    b, c = len(lengths), H * P
    td, tol = TD[dtype], {"bf16": 2e-2, "fp32": 1e-4}[dtype]
    g = torch.Generator().manual_seed(65)
    rnd = lambda *s: torch.randn(*s, generator=g)
    past = torch.arange(L)[None, :] >= torch.tensor(lengths)[:, None]
    xbc, z = rnd(b, L, c + 2 * N).to(td), rnd(b, L, c).to(td)
    dt = torch.nn.functional.softplus(rnd(b, L, H) - 4).to(td)
    dt[past] = 0
    w, bias = 0.5 * rnd(c + 2 * N, 4), 0.1 * rnd(c + 2 * N)
    A, D, nw = -torch.exp(rnd(H)), torch.rand(H, generator=g), 1 + 0.1 * rnd(c)
    noisy = xbc.clone()
    noisy[past] = float("nan")              # what stands behind a sequence is not read
    lt = torch.tensor(lengths, dtype=torch.int32, device=dev)
    _fill_free_memory(dev, td, b * L * c, b * L * N, b * L * (c + 2 * N))
    (x, B, C), cs = ssd.ssd_conv(noisy.to(dev), w.to(dev), bias.to(dev), lengths=lt, split=[c, N, N])
    y, hT = ssd.ssd_forward(x.view(b, L, H, P), dt.to(dev), A.to(dev), B.view(b, L, 1, N),
                            C.view(b, L, 1, N), D.to(dev), chunk=64)
    out = ssd.ssd_norm(y.view(b, L, c), nw.to(dev), z.to(dev))
    torch.cuda.synchronize()

    for i, m in enumerate(lengths):
        v, _, fin = ref.conv(xbc[i:i + 1, :m], w, bias, None, None, True)
        rep = lambda t: t.double().repeat_interleave(P, -1)
        yr, _, hr, _ = ref.scan(v[..., :c], rep(dt[i:i + 1, :m]), rep(A)[:, None].expand(c, N),
                                v[..., None, c:c + N], v[..., None, c + N:], rep(D))
        yo, _, _, _ = ref.norm(yr[0], nw, z[i, :m])
        for got, want, what in ((out[i, :m], yo, "out"), (hT[i].view(c, N), hr[0], "state"),
                                (cs[i], fin[0], "conv state")):
            err = ((ref.d64(got) - want).abs().max() / want.abs().max()).item()
            print(f"  sequence {i}, {what}: {err:.2e}", flush=True)
            assert err <= tol, (i, what, err)
