"""Host-side checks of the operators around the forward (short convolution, selective scan,
block norms): every refusal comes before any launch.  No GPU needed."""
import ctypes

import pytest
import torch

import state_space_sequence_cumsum_amd as ssd
from state_space_sequence_cumsum_amd import binding, block

OK16 = ctypes.c_void_p(4096)      # never dereferenced: validation fails first
OFF4 = ctypes.c_void_p(4096 + 4)
OFF2 = ctypes.c_void_p(4096 + 2)


def _conv(**kw):
    base = dict(batch=2, seqlen=100, channels=320, x_pitch=0, split=(192, 64, 64), width=4, silu=1,
                dtype=1)
    base.update(kw)
    base["split"] = (ctypes.c_int64 * 3)(*base["split"])
    return ssd.ConvProblem(**base)


def _scan(**kw):
    base = dict(batch=2, seqlen=100, channels=256, ngroups=2, dstate=16, x_pitch=0, dt_pitch=0,
                z_pitch=0, B_pitch=0, C_pitch=0, softplus=1, dtype=1)
    base.update(kw)
    return ssd.ScanProblem(**base)


def _norm(**kw):
    base = dict(rows=10, channels=256, ngroups=2, x_pitch=0, z_pitch=0, eps=1e-5, scale=1.0,
                gate_after=0, dtype=1, residual_dtype=0)
    base.update(kw)
    return ssd.NormProblem(**base)


def test_every_entry_point_is_declared_and_exported():
    names = {"ssd_conv", "ssd_conv_step", "ssd_conv_validate", "ssd_scan", "ssd_scan_step",
             "ssd_scan_validate", "ssd_scan_workspace_bytes", "ssd_norm", "ssd_norm_validate"}
    assert names <= set(binding.header_functions())
    assert all(hasattr(block.lib(), n) for n in names)


@pytest.mark.parametrize("kw,status", [
    (dict(), 0),
    (dict(x_pitch=320), 0),
    (dict(x_pitch=1001), 0),
    (dict(channels=5, split=(5, 0, 0)), 0),
    (dict(batch=0), 2),
    (dict(seqlen=0), 2),
    (dict(channels=-1), 2),
    (dict(split=(192, 64, 63)), 2),
    (dict(split=(320, 0, 1)), 2),
    (dict(split=(256, 0, 64)), 2),
    (dict(split=(0, 256, 64)), 2),
    (dict(split=(1 << 62, 1 << 62, 320 - (1 << 62))), 2),
    (dict(x_pitch=319), 2),
    (dict(x_pitch=-320), 2),
    (dict(width=1), 3),
    (dict(width=5), 3),
    (dict(dtype=2), 3),
    (dict(silu=2), 3),
    (dict(x_pitch=(1 << 24) + 1), 3),
    (dict(seqlen=(1 << 30) + 1), 3),
    (dict(batch=1 << 22, seqlen=1 << 10), 3),
    (dict(batch=(1 << 24) // 2 - 1, seqlen=8), 0),
    (dict(batch=(1 << 24) // 2, seqlen=8), 3),
    (dict(batch=1 << 40), 3),
])
def test_conv_validate(kw, status):
    p = _conv(**kw)
    assert block.lib().ssd_conv_validate(ctypes.byref(p)) == status
    if status:      # the entry points refuse the same problems
        a = [OK16] * 10
        assert block.lib().ssd_conv(ctypes.byref(p), *a[:9], None) == status
        assert block.lib().ssd_conv_step(ctypes.byref(p), *a[:7], None) == status


def test_conv_pointer_checks():
    L, p = block.lib(), _conv()
    # x, weight, bias, state0, lengths, y0, y1, y2, stateT, stream
    for missing in (0, 1, 5, 6, 7):
        a = [OK16] * 9
        a[missing] = None
        assert L.ssd_conv(ctypes.byref(p), *a, None) == 1
    for off in (1, 2):
        a = [OK16] * 9
        a[off] = OFF4
        assert L.ssd_conv(ctypes.byref(p), *a, None) == 6
    s = _conv(seqlen=1)
    assert L.ssd_conv_step(ctypes.byref(_conv(seqlen=2)), *[OK16] * 7, None) == 2
    for missing in (0, 1, 3, 4, 5, 6):
        a = [OK16] * 7
        a[missing] = None
        assert L.ssd_conv_step(ctypes.byref(s), *a, None) == 1
    assert L.ssd_conv_step(ctypes.byref(s), OK16, OFF4, *[OK16] * 5, None) == 6
    for fn, n in ((L.ssd_conv, 9), (L.ssd_conv_step, 7)):
        assert fn(None, *[OK16] * n, None) == 1
    assert L.ssd_conv_validate(None) == 1
    assert binding.lib().ssd_last_hip_error() == 0


@pytest.mark.parametrize("kw,status", [
    (dict(), 0),
    (dict(dstate=64, ngroups=256), 0),
    (dict(B_pitch=33, C_pitch=100, z_pitch=256, x_pitch=300, dt_pitch=257), 0),
    (dict(batch=0), 2),
    (dict(seqlen=0), 2),
    (dict(channels=0), 2),
    (dict(ngroups=3), 2),
    (dict(ngroups=0), 2),
    (dict(dstate=-8), 2),
    (dict(x_pitch=255), 2),
    (dict(dt_pitch=-1), 2),
    (dict(z_pitch=100), 2),
    (dict(B_pitch=31), 2),
    (dict(C_pitch=16), 2),
    (dict(dstate=12), 3),
    (dict(dstate=72), 3),
    (dict(dtype=-1), 3),
    (dict(softplus=7), 3),
    (dict(channels=1 << 25), 3),
    (dict(z_pitch=1 << 29), 3),
    (dict(seqlen=1 << 31), 3),
    (dict(batch=1 << 12, seqlen=1 << 20), 3),
    (dict(batch=1 << 20), 3),
    (dict(batch=1 << 40, seqlen=1), 3),
    (dict(batch=(1 << 20) // 4 - 1, seqlen=1), 0),
])
def test_scan_validate(kw, status):
    L, p = block.lib(), _scan(**kw)
    assert L.ssd_scan_validate(ctypes.byref(p)) == status
    assert (ssd.ssd_scan_workspace_bytes(p) > 0) == (status == 0)
    if status:
        assert L.ssd_scan(ctypes.byref(p), *[OK16] * 13, 1 << 50, None) == status
        assert L.ssd_scan_step(ctypes.byref(p), *[OK16] * 10, None) == status


def test_scan_pointer_checks():
    L, p = block.lib(), _scan()
    n = ssd.ssd_scan_workspace_bytes(p)
    # x, dt, A, B, C, D, z, dt_bias, h0, lengths, y, hT, workspace
    for missing in (0, 1, 2, 3, 4, 10):
        a = [OK16] * 13
        a[missing] = None
        assert L.ssd_scan(ctypes.byref(p), *a, n, None) == 1
    # short prompts and whole walks take no workspace; segments do
    assert n == 1 and ssd.ssd_scan_workspace_bytes(_scan(batch=512)) == 1
    assert "#define SSD_SCAN_NO_WORKSPACE 1u" in open(binding.HEADER).read()
    long = _scan(seqlen=1000)
    n = ssd.ssd_scan_workspace_bytes(long)
    assert n > 1000
    assert L.ssd_scan(ctypes.byref(long), *[OK16] * 13, n - 1, None) == 4
    assert L.ssd_scan(ctypes.byref(long), *[OK16] * 12, None, n, None) == 4
    for off, ptr in ((2, OFF4), (8, OFF4), (11, OFF4), (12, OFF4), (3, OFF2), (4, OFF2)):
        a = [OK16] * 13
        a[off] = ptr
        assert L.ssd_scan(ctypes.byref(p), *a, n, None) == 6
    # bf16 B and C rows are read as dwords; fp32 rows always are
    assert L.ssd_scan(ctypes.byref(_scan(B_pitch=33)), *[OK16] * 13, 1 << 40, None) == 6
    assert L.ssd_scan(ctypes.byref(_scan(C_pitch=33)), *[OK16] * 13, 1 << 40, None) == 6
    s = _scan(seqlen=1)
    # x, dt, A, B, C, D, z, dt_bias, h, y
    assert L.ssd_scan_step(ctypes.byref(p), *[OK16] * 10, None) == 2
    for missing in (0, 1, 2, 3, 4, 8, 9):
        a = [OK16] * 10
        a[missing] = None
        assert L.ssd_scan_step(ctypes.byref(s), *a, None) == 1
    for off, ptr in ((2, OFF4), (8, OFF4), (3, OFF2), (4, OFF2)):
        a = [OK16] * 10
        a[off] = ptr
        assert L.ssd_scan_step(ctypes.byref(s), *a, None) == 6
    assert L.ssd_scan_validate(None) == 1 and L.ssd_scan_workspace_bytes(None) == 0
    assert binding.lib().ssd_last_hip_error() == 0


@pytest.mark.parametrize("kw,status", [
    (dict(), 0),
    (dict(dtype=0), 0),
    (dict(residual_dtype=1), 0),
    (dict(x_pitch=300, z_pitch=256), 0),
    (dict(rows=0), 2),
    (dict(channels=0), 2),
    (dict(ngroups=3), 2),
    (dict(ngroups=-2), 2),
    (dict(x_pitch=255), 2),
    (dict(z_pitch=-4), 2),
    (dict(dtype=3), 3),
    (dict(dtype=0, residual_dtype=1), 3),
    (dict(gate_after=2), 3),
    (dict(eps=0.0), 3),
    (dict(eps=-1.0), 3),
    (dict(eps=float("nan")), 3),
    (dict(eps=float("inf")), 3),
    (dict(scale=float("nan")), 3),
    (dict(scale=float("inf")), 3),
    (dict(channels=1 << 25), 3),
    (dict(z_pitch=1 << 29), 3),
    (dict(rows=1 << 23), 3),
    (dict(rows=(1 << 23) - 1), 0),
    (dict(rows=1 << 62, ngroups=1), 3),
])
def test_norm_validate(kw, status):
    L, p = block.lib(), _norm(**kw)
    assert L.ssd_norm_validate(ctypes.byref(p)) == status
    if status:
        assert L.ssd_norm(ctypes.byref(p), *[OK16] * 6, None) == status


@pytest.mark.parametrize("eps,status", [
    (2.0 ** -126, 0), (1e-30, 0), (1e30, 0), (2.0 ** -127, 3), (1e-39, 3), (1e-45, 3), (1e-60, 3)])
def test_norm_eps_is_a_normal_number(eps, status):
    """A row of zeros has eps alone under its root, which takes a subnormal number for zero."""
    assert block.lib().ssd_norm_validate(ctypes.byref(_norm(eps=eps))) == status


def test_norm_pointer_checks():
    L, p = block.lib(), _norm()
    # x, z, residual, weight, y, residual_out
    for missing in (0, 2, 3, 4):
        a = [OK16] * 6
        a[missing] = None
        assert L.ssd_norm(ctypes.byref(p), *a, None) == 1      # 2: residual_out without a residual
    assert L.ssd_norm(ctypes.byref(p), *[OK16] * 3, OFF4, OK16, OK16, None) == 6
    assert L.ssd_norm(None, *[OK16] * 6, None) == 1 and L.ssd_norm_validate(None) == 1
    assert binding.lib().ssd_last_hip_error() == 0


def test_binding_refuses_host_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ssd.ssd_conv(bf(1, 4, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError):
        ssd.ConvStepPlan(bf(1, 8), torch.zeros(8, 4), None, bf(1, 3, 8))
    with pytest.raises(ValueError):
        ssd.ssd_scan(bf(1, 4, 8), bf(1, 4, 8), torch.zeros(8, 16), bf(1, 4, 1, 16), bf(1, 4, 1, 16))
    with pytest.raises(ValueError):
        ssd.ScanStepPlan(bf(1, 8), bf(1, 8), torch.zeros(8, 16), bf(1, 1, 16), bf(1, 1, 16),
                         torch.zeros(1, 8, 16))
    with pytest.raises(ValueError):
        ssd.ssd_norm(bf(4, 8), torch.zeros(8))
    for t in (torch.zeros(4, 8, dtype=torch.float16), None, 3):
        with pytest.raises(ValueError):
            ssd.ssd_norm(t, torch.zeros(8))


@pytest.mark.parametrize("shape,stride,lead,pitch", [
    ((2, 5, 8), (40, 8, 1), 2, 8),
    ((2, 5, 8), (100, 20, 1), 2, 20),
    ((2, 1, 8), (20, 7, 1), 2, 20),       # one token: the batch stride is the pitch
    ((1, 5, 8), (3, 20, 1), 2, 20),       # one sequence: its stride is not used
    ((1, 1, 8), (1, 1, 1), 2, 0),
    ((2, 5, 1, 16), (160, 32, 9, 1), 2, 32),
    ((2, 5, 2, 16), (160, 32, 16, 1), 2, 32),
    ((6, 8), (8, 1), 1, 8),
    ((6, 1), (4, 3), 1, 4),
    ((2, 5, 8), (80, 8, 1), 2, None),     # tokens of the next batch not where they belong
    ((2, 5, 8), (40, 8, 2), 2, None),     # channels not dense
    ((2, 5, 2, 16), (320, 64, 32, 1), 2, None),
    ((2, 5, 8), (0, 8, 1), 2, None),      # expanded
    ((2, 5, 8), (20, 4, 1), 2, None),     # rows that overlap
    ((6, 8), (0, 1), 1, None),
])
def test_row_layouts(shape, stride, lead, pitch):
    t = torch.empty(4096).as_strided(shape, stride)
    if pitch is None:
        with pytest.raises(ValueError):
            block._pitch(t, "t", lead)
    else:
        assert block._pitch(t, "t", lead) == pitch


# ---------------------------------------------------------------------------
# outputs apart from the other arguments: addresses far apart, but for the pair under test
# (every call here is refused, so none of them is ever read)
# ---------------------------------------------------------------------------
def _far(n):
    return [(i + 1) << 40 for i in range(n)]


def _refused(fn, problem, ptrs, *tail):
    args = [ctypes.c_void_p(p) for p in ptrs]
    return fn(ctypes.byref(problem), *args, *tail, None) == 9


def test_overlap_has_a_status():
    assert "memory" in ssd.ssd_status_string(9) and binding.STATUS[9] == "SSD_ERR_OVERLAP"


@pytest.mark.parametrize("out,other,off", [
    (5, 0, 0),                     # y0 on x: a later token tile would read replaced rows
    (5, 0, 200 * 320 * 2 - 16), (5, 0, 16 - 200 * 192 * 2),     # x's last and first 16 bytes
    (6, 0, 4096), (7, 0, 64), (8, 0, 0), (5, 1, 0), (6, 2, 0), (7, 3, 0), (7, 4, 0), (6, 5, 0),
    (7, 5, 256), (7, 6, 16), (8, 5, 0), (8, 7, 0), (8, 1, 0),
    (8, 3, 16),                    # the final state in the state's buffer, but not at its start
])
def test_conv_outputs_apart(out, other, off):
    # x, weight, bias, state0, lengths, y0, y1, y2, stateT
    a = _far(9)
    a[out] = a[other] + off
    assert _refused(block.lib().ssd_conv, _conv(), a)


def test_conv_output_between_rows_of_x():
    """Rows of x are 320 of 1000 elements: what reaches into a row is refused."""
    p = _conv(x_pitch=1000, batch=1, seqlen=3, split=(320, 0, 0))
    a = _far(9)
    for off in (638, 2000 - 1918, 2000, 2000 + 638, 2 * 2000 + 638, -2):
        a[5] = a[0] + off
        assert _refused(block.lib().ssd_conv, p, a), off


@pytest.mark.parametrize("out,other,off", [
    (4, 0, 2), (5, 0, 0), (6, 0, 0), (3, 0, 0), (3, 1, 0), (4, 1, 0), (5, 2, 0), (5, 3, 2), (5, 4, 64),
    (4, 0, 0),                     # y0 at x's start, but narrower rows
])
def test_conv_step_outputs_apart(out, other, off):
    # x, weight, bias, state, y0, y1, y2
    a = _far(7)
    a[out] = a[other] + off
    assert _refused(block.lib().ssd_conv_step, _conv(seqlen=1), a)
    # one output on a wider array's rows
    a = _far(7)
    a[4] = a[0]
    assert _refused(block.lib().ssd_conv_step,
                    _conv(seqlen=1, split=(320, 0, 0), x_pitch=328), a)


@pytest.mark.parametrize("out,other,off", [
    (10, 0, 0), (10, 1, 0), (10, 6, 0), (10, 3, 64), (10, 4, 0), (10, 2, 0), (10, 5, 0), (10, 7, 16),
    (10, 8, 0), (10, 9, 0), (10, 11, 0), (10, 12, 0), (11, 0, 0), (11, 2, 0), (11, 8, 16), (11, 12, 0),
    (12, 0, 0), (12, 8, 0), (12, 4, 1024), (11, 9, 0)])
def test_scan_outputs_apart(out, other, off):
    # x, dt, A, B, C, D, z, dt_bias, h0, lengths, y, hT, workspace
    p = _scan(seqlen=1000)
    a = _far(13)
    a[out] = a[other] + off
    assert _refused(block.lib().ssd_scan, p, a, ctypes.c_size_t(1 << 30))


@pytest.mark.parametrize("out,other,off", [
    (9, 0, 2), (9, 1, 16), (9, 6, -2), (9, 3, 0), (9, 4, 0), (9, 2, 0), (9, 8, 0), (8, 0, 0), (8, 2, 0),
    (8, 4, 0), (8, 5, 0)])
def test_scan_step_outputs_apart(out, other, off):
    # x, dt, A, B, C, D, z, dt_bias, h, y
    a = _far(10)
    a[out] = a[other] + off
    assert _refused(block.lib().ssd_scan_step, _scan(seqlen=1), a)
    # groups so many that y and B are of one size: B's rows are still not y's
    a = _far(10)
    a[9] = a[3]
    assert _refused(block.lib().ssd_scan_step, _scan(seqlen=1, channels=256, ngroups=16), a)


@pytest.mark.parametrize("kw,out,other,off", [
    ({}, 4, 0, 2), ({}, 4, 1, 512), ({}, 4, 3, 0), ({}, 5, 3, 0), ({}, 4, 5, 0), ({}, 5, 4, 0),
    ({}, 4, 2, 0),                 # bf16 rows in a fp32 residual's buffer
    ({}, 5, 0, 0),                 # and the other way round
    (dict(residual_dtype=1), 5, 2, 16),
    (dict(x_pitch=264), 4, 0, 0), (dict(z_pitch=512), 4, 1, 0)])
def test_norm_outputs_apart(kw, out, other, off):
    # x, z, residual, weight, y, residual_out
    a = _far(6)
    a[out] = a[other] + off
    assert _refused(block.lib().ssd_norm, _norm(**kw), a)
