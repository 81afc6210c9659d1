"""Host-side checks of linear attention and rotary positions: every refusal comes before any launch;
and the 64-bit references of their GPU tests against the recurrence itself.  No GPU needed."""
import ctypes
import math

import pytest
import torch

import linattn_ref as ref
import state_space_sequence_cumsum_amd as ssd
from state_space_sequence_cumsum_amd import binding, linattn

OK16 = ctypes.c_void_p(4096)      # never dereferenced: validation fails first
OFF8 = ctypes.c_void_p(4096 + 8)
OFF2 = ctypes.c_void_p(4096 + 2)
OFF1 = ctypes.c_void_p(4096 + 1)


def _problem(**kw):
    base = dict(batch=2, seqlen=100, nheads=8, ngroups=4, key_dim=64, value_dim=128, q_pitch=0,
                k_pitch=0, v_pitch=0, g_pitch=0, do_pitch=0, scale=1.0, decay=2, dtype=1)
    base.update(kw)
    return ssd.LinattnProblem(**base)


def _rotary(**kw):
    base = dict(batch=2, seqlen=100, q_heads=8, k_heads=4, head_dim=64, rotated=64, q_pitch=0,
                k_pitch=0, scale=1.0, positions=1, interleaved=0, inverse=0, dtype=1)
    base.update(kw)
    return ssd.RotaryProblem(**base)


def test_every_entry_point_is_declared_and_exported():
    names = {"ssd_linattn", "ssd_linattn_step", "ssd_linattn_validate",
             "ssd_linattn_workspace_bytes", "ssd_linattn_backward",
             "ssd_linattn_backward_workspace_bytes", "ssd_rotary", "ssd_rotary_validate"}
    assert names <= set(binding.header_functions())
    assert all(hasattr(linattn.lib(), n) for n in names)


LINATTN_PROBLEMS = [
    (dict(), 0),
    (dict(key_dim=8, value_dim=256), 0),
    (dict(q_pitch=256, k_pitch=264, v_pitch=1 << 22, g_pitch=9, do_pitch=1024), 0),
    (dict(decay=0), 0),
    (dict(decay=1, g_pitch=3), 0),
    (dict(scale=-0.5), 0),
    (dict(scale=0.0), 0),
    (dict(batch=65535, nheads=1, ngroups=1), 0),
    (dict(batch=0), 2),
    (dict(seqlen=0), 2),
    (dict(nheads=-8), 2),
    (dict(ngroups=3), 2),
    (dict(ngroups=0), 2),
    (dict(key_dim=0), 2),
    (dict(value_dim=-8), 2),
    (dict(q_pitch=255), 2),
    (dict(k_pitch=-256), 2),
    (dict(v_pitch=1023), 2),
    (dict(do_pitch=8), 2),
    (dict(g_pitch=7), 2),
    (dict(key_dim=12), 3),
    (dict(key_dim=264), 3),
    (dict(value_dim=264), 3),
    (dict(value_dim=4), 3),
    (dict(dtype=2), 3),
    (dict(decay=3), 3),
    (dict(decay=-1), 3),
    (dict(scale=math.inf), 3),
    (dict(scale=math.nan), 3),
    (dict(batch=8192), 3),
    (dict(batch=1 << 60), 3),
    (dict(nheads=1 << 40, ngroups=1 << 40), 3),
    (dict(q_pitch=(1 << 22) + 8), 3),
    (dict(v_pitch=1 << 40), 3),
    (dict(seqlen=(1 << 30) + 1), 3),
    (dict(seqlen=1 << 30, batch=3), 3),
]


@pytest.mark.parametrize("kw,status", LINATTN_PROBLEMS)
def test_linattn_validate(kw, status):
    L, p = linattn.lib(), _problem(**kw)
    assert L.ssd_linattn_validate(ctypes.byref(p)) == status
    assert (ssd.ssd_linattn_workspace_bytes(p) > 0) == (status == 0)
    if status:      # the entry points refuse the same problems
        assert L.ssd_linattn(ctypes.byref(p), *[OK16] * 9, 1 << 50, None) == status
        assert L.ssd_linattn_step(ctypes.byref(p), *[OK16] * 6, None) == status
        assert L.ssd_linattn_backward(ctypes.byref(p), *[OK16] * 14, 1 << 50, None) == status
    assert (ssd.ssd_linattn_backward_workspace_bytes(p) > 0) == (status == 0)


def test_gradient_pointer_checks():
    L, p = linattn.lib(), _problem()
    n = ssd.ssd_linattn_backward_workspace_bytes(p)
    assert n > 1 and ssd.ssd_linattn_backward_workspace_bytes(_problem(ngroups=8, decay=1)) == 1
    # do, q, k, v, g, h0, dhT, lengths, dq, dk, dv, dg, dh0, workspace
    for missing in (0, 1, 2, 3, 4, 8, 9, 10):
        a = [OK16] * 14
        a[missing] = None
        assert L.ssd_linattn_backward(ctypes.byref(p), *a, n, None) == 1
    assert L.ssd_linattn_backward(ctypes.byref(p), *[OK16] * 13, None, n, None) == 4
    assert L.ssd_linattn_backward(ctypes.byref(p), *[OK16] * 14, n - 1, None) == 4
    for off in (0, 1, 2, 3, 5, 6, 8, 9, 10, 12, 13):
        a = [OK16] * 14
        a[off] = OFF8
        assert L.ssd_linattn_backward(ctypes.byref(p), *a, n, None) == 6
    for pitch in ("q_pitch", "k_pitch", "v_pitch", "do_pitch"):
        assert L.ssd_linattn_backward(ctypes.byref(_problem(**{pitch: 1028})), *[OK16] * 14, 1 << 40, None) == 6
    # decays that are not given per token have no gradient
    for decay in (0, 1):
        assert L.ssd_linattn_backward(ctypes.byref(_problem(decay=decay)), *[OK16] * 14, n, None) == 3
    assert L.ssd_linattn_backward(None, *[OK16] * 14, n, None) == 1
    assert L.ssd_linattn_backward_workspace_bytes(None) == 0


@pytest.mark.parametrize("out", [8, 9, 10, 11, 12, 13])
def test_gradient_outputs_apart(out):
    # do, q, k, v, g, h0, dhT, lengths, dq, dk, dv, dg, dh0, workspace
    for other in range(14):
        if other != out:
            a = _far(14)
            a[out] = a[other]
            assert _refused(linattn.lib().ssd_linattn_backward, _problem(), a, ctypes.c_size_t(1 << 40))


def test_linattn_pointer_checks():
    L, p = linattn.lib(), _problem()
    # q, k, v, g, h0, lengths, o, hT, workspace
    for missing in (0, 1, 2, 3, 6):
        a = [OK16] * 9
        a[missing] = None
        assert L.ssd_linattn(ctypes.byref(p), *a, 1 << 50, None) == 1
    for off in (0, 1, 2, 4, 6, 7):
        a = [OK16] * 9
        a[off] = OFF8
        assert L.ssd_linattn(ctypes.byref(p), *a, 1 << 50, None) == 6
    for pitch in ("q_pitch", "k_pitch", "v_pitch"):
        bad = _problem(**{pitch: 1028})
        assert L.ssd_linattn(ctypes.byref(bad), *[OK16] * 9, 1 << 50, None) == 6
        assert L.ssd_linattn_step(ctypes.byref(_problem(seqlen=1, **{pitch: 1028})), *[OK16] * 6, None) == 6
    s = _problem(seqlen=1)
    # q, k, v, g, h, o
    assert L.ssd_linattn_step(ctypes.byref(p), *[OK16] * 6, None) == 2
    for missing in range(6):
        a = [OK16] * 6
        a[missing] = None
        assert L.ssd_linattn_step(ctypes.byref(s), *a, None) == 1
    for off in (0, 1, 2, 4, 5):
        a = [OK16] * 6
        a[off] = OFF8
        assert L.ssd_linattn_step(ctypes.byref(s), *a, None) == 6
    assert L.ssd_linattn_validate(None) == 1 and L.ssd_linattn_workspace_bytes(None) == 0
    assert L.ssd_linattn(None, *[OK16] * 9, 0, None) == 1
    assert L.ssd_linattn_step(None, *[OK16] * 6, None) == 1
    assert "#define SSD_LINATTN_NO_WORKSPACE 1u" in open(binding.HEADER).read()
    assert binding.lib().ssd_last_hip_error() == 0


def test_decays_and_lengths_on_their_own_sizes():
    L, odd = linattn.lib(), ctypes.c_void_p(OK16.value + 2 + 1)
    for decay, dtype in ((1, 1), (2, 0), (2, 1)):
        kw = dict(decay=decay, dtype=dtype)
        for at in (3, 5):                            # g, lengths
            a = [OK16] * 9
            a[at] = odd
            assert L.ssd_linattn(ctypes.byref(_problem(**kw)), *a, 1 << 50, None) == 6
        a = [OK16] * 6
        a[3] = odd
        assert L.ssd_linattn_step(ctypes.byref(_problem(seqlen=1, **kw)), *a, None) == 6
        for at in (4, 7) + ((11,) if decay == 2 else ()):
            a = [OK16] * 14
            a[at] = odd
            if decay != 2:
                a[11] = None
            assert L.ssd_linattn_backward(ctypes.byref(_problem(**kw)), *a, 1 << 50, None) == 6


def _far(n):
    return [(i + 1) << 40 for i in range(n)]


def _refused(fn, problem, ptrs, *tail):
    args = [ctypes.c_void_p(p) for p in ptrs]
    return fn(ctypes.byref(problem), *args, *tail, None) == 9


@pytest.mark.parametrize("out,other,off", [
    (6, 0, 0), (6, 1, 64), (6, 2, 0), (6, 3, 0), (6, 4, 0), (6, 5, 0), (6, 7, 0), (7, 0, 0), (7, 2, 16),
    (7, 3, 0), (7, 5, 0),
    (7, 4, 16),                    # the final state in the initial one's buffer, but not at its start
])
def test_linattn_outputs_apart(out, other, off):
    # q, k, v, g, h0, lengths, o, hT, workspace
    a = _far(9)
    a[out] = a[other] + off
    assert _refused(linattn.lib().ssd_linattn, _problem(), a, ctypes.c_size_t(1 << 40))


@pytest.mark.parametrize("out,other,off", [
    (5, 0, 0), (5, 1, 0), (5, 3, 0), (5, 4, 0), (5, 2, 16), (4, 0, 0), (4, 2, 0), (4, 3, 0)])
def test_linattn_step_outputs_apart(out, other, off):
    # q, k, v, g, h, o
    a = _far(6)
    a[out] = a[other] + off
    assert _refused(linattn.lib().ssd_linattn_step, _problem(seqlen=1), a)
    a = _far(6)
    a[5] = a[2]                    # one output on a wider array's rows
    assert _refused(linattn.lib().ssd_linattn_step, _problem(seqlen=1, v_pitch=2048), a)


@pytest.mark.parametrize("kw,status", [
    (dict(), 0),
    (dict(k_heads=0), 0),
    (dict(head_dim=33, rotated=2), 0),
    (dict(q_pitch=513, k_pitch=300), 0),
    (dict(positions=0), 0),
    (dict(scale=0.0), 0),
    (dict(batch=0), 2),
    (dict(seqlen=-1), 2),
    (dict(q_heads=0), 2),
    (dict(k_heads=-1), 2),
    (dict(head_dim=0), 2),
    (dict(rotated=0), 2),
    (dict(rotated=66), 2),
    (dict(rotated=63), 2),
    (dict(q_pitch=511), 2),
    (dict(k_pitch=-1), 2),
    (dict(head_dim=8192), 3),
    (dict(q_heads=1 << 17), 3),
    (dict(k_heads=1 << 60), 3),
    (dict(dtype=5), 3),
    (dict(scale=math.inf), 3),
    (dict(interleaved=2), 3),
    (dict(inverse=-1), 3),
    (dict(positions=3), 3),
    (dict(q_pitch=(1 << 22) + 1), 3),
    (dict(batch=1 << 12, seqlen=1 << 12), 3),
    (dict(batch=1 << 40), 3),
])
def test_rotary_validate(kw, status):
    L, p = linattn.lib(), _rotary(**kw)
    assert L.ssd_rotary_validate(ctypes.byref(p)) == status
    if status:
        assert L.ssd_rotary(ctypes.byref(p), *[OK16] * 6, None) == status


def test_rotary_pointer_checks():
    L, p = linattn.lib(), _rotary()
    # q, k, freqs, positions, q_out, k_out
    for missing in range(6):
        a = [OK16] * 6
        a[missing] = None
        assert L.ssd_rotary(ctypes.byref(p), *a, None) == 1
    for off, ptr in ((0, OFF1), (1, OFF1), (2, OFF2), (3, OFF2), (4, OFF1), (5, OFF1)):
        a = [OK16] * 6
        a[off] = ptr
        assert L.ssd_rotary(ctypes.byref(p), *a, None) == 6
    assert L.ssd_rotary(None, *[OK16] * 6, None) == 1 and L.ssd_rotary_validate(None) == 1


@pytest.mark.parametrize("kw,out,other,off", [
    ({}, 4, 0, 2), ({}, 4, 1, 0), ({}, 4, 2, 0), ({}, 4, 3, 0), ({}, 4, 5, 0), ({}, 5, 0, 0), ({}, 5, 1, 16),
    ({}, 5, 2, 0), ({}, 5, 3, 0), (dict(q_pitch=600), 4, 0, 0), (dict(k_pitch=512), 5, 1, 0)])
def test_rotary_outputs_apart(kw, out, other, off):
    a = _far(6)
    a[out] = a[other] + off
    assert _refused(linattn.lib().ssd_rotary, _rotary(**kw), a)


def test_binding_refuses_host_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, v = bf(1, 4, 2, 8), bf(1, 4, 2, 8)
    with pytest.raises(ValueError):
        ssd.ssd_linattn(q, q, v)
    with pytest.raises(ValueError):
        ssd.LinattnStepPlan(q[:, 0], q[:, 0], v[:, 0], torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError):
        ssd.ssd_linattn_backward(v, q, q, v)
    with pytest.raises(ValueError):
        ssd.ssd_rotary(q, None, torch.ones(4))
    for t in (torch.zeros(1, 4, 2, 8, dtype=torch.float16), None, 3):
        with pytest.raises(ValueError):
            ssd.ssd_linattn(t, q, v)
        with pytest.raises(ValueError):
            ssd.ssd_rotary(t, None, torch.ones(4))


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def test_rotary_frequencies():
    f = ssd.rotary_frequencies(8, 10000.0)
    assert f.dtype == torch.float32 and torch.equal(f, torch.tensor([1.0, 0.1, 0.01, 0.001]))
    assert torch.equal(ssd.rotary_frequencies(8, scaling="linear", factor=4.0), f / 4)
    grown = ssd.rotary_frequencies(8, scaling="base", factor=4.0)
    assert grown[0] == 1.0 and math.isclose(grown[3], 0.001 / 4, rel_tol=1e-6)
    # 1000 tokens: the first pair turns 159 times, the third 1.6 times, the last 0.16 times
    parts = ssd.rotary_frequencies(8, scaling="parts", factor=4.0, length=1000)
    assert parts[0] == 1.0 and parts[3] == 0.001 / 4
    keep = (1000 * 0.01 / (2 * math.pi) - 1) / 31
    assert math.isclose(parts[2], 0.01 * keep + 0.01 / 4 * (1 - keep), rel_tol=1e-6)


@pytest.mark.parametrize("args,kw", [
    ((7,), {}), ((0,), {}), ((8,), dict(factor=0.0)), ((8, -1.0), {}), ((2,), dict(scaling="base", factor=2.0)),
    ((8,), dict(scaling="parts", factor=2.0)), ((8,), dict(scaling="parts", length=10, slow=4, fast=4)),
    ((8,), dict(scaling="other"))])
def test_rotary_frequencies_refusals(args, kw):
    with pytest.raises(ValueError):
        ssd.rotary_frequencies(*args, **kw)


# ---------------------------------------------------------------------------
# the references of the GPU tests against the recurrence, token by token
# ---------------------------------------------------------------------------
def _recurrence(q, k, v, g, S, scale):
    """Inputs [b, L, H, w] (one head of q and k for each of v), g [b, L, H] -> (o, S)."""
    outs = []
    for t in range(q.shape[1]):
        S = S * g[:, t, :, None, None].exp() + v[:, t, :, :, None] * k[:, t, :, None, :]
        outs.append(scale * (S * q[:, t, :, None, :]).sum(3))
    return torch.stack(outs, 1), S


@pytest.mark.parametrize("L,G,H", [(1, 1, 1), (70, 2, 2), (130, 1, 3)])
def test_references_match_the_recurrence_and_its_gradients(L, G, H):
    gen = torch.Generator().manual_seed(L)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    b, dk, dv, scale = 2, 3, 5, 0.7
    q, k, v, do = rnd(b, L, G, dk), rnd(b, L, G, dk), rnd(b, L, H, dv), rnd(b, L, H, dv)
    g, h0, dhT = -rnd(b, L, H).abs(), rnd(b, H, dv, dk), rnd(b, H, dv, dk)
    leaves = [t.requires_grad_() for t in (q, k, v, g, h0)]
    wide = lambda t: t.repeat_interleave(H // G, 2)
    o, S = _recurrence(wide(q), wide(k), v, g, h0, scale)
    grads = torch.autograd.grad((o * do).sum() + (S * dhT).sum(), leaves)
    ro, _, rS, _ = ref.forward(q, k, v, g, h0, scale)
    got = ref.backward(do, q, k, v, g, h0, dhT, scale)
    for x, y in [(o, ro), (S, rS)] + [(x, y[0]) for x, y in zip(grads, got)]:
        assert torch.allclose(x, y, rtol=1e-10, atol=1e-10)


def test_gradient_references_match_differences():
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    b, L, G, H, dk, dv, scale = 1, 66, 1, 2, 3, 2, 0.5
    args = dict(q=rnd(b, L, G, dk), k=rnd(b, L, G, dk), v=rnd(b, L, H, dv), g=-rnd(b, L, H).abs(),
                h0=rnd(b, H, dv, dk))
    do, dhT = rnd(b, L, H, dv), rnd(b, H, dv, dk)
    value = lambda a: sum((x * y).sum() for x, y in zip(ref.forward(**a, scale=scale)[::2], (do, dhT)))
    got = ref.backward(do, **args, dhT=dhT, scale=scale)
    for name, (grad, _) in zip(("q", "k", "v", "g", "h0"), got):
        direction = rnd(*args[name].shape)
        up, down = ({**args, name: args[name] + e * direction} for e in (1e-6, -1e-6))
        slope = (value(up) - value(down)) / 2e-6
        assert math.isclose(slope, (grad * direction).sum(), rel_tol=1e-6, abs_tol=1e-6)
