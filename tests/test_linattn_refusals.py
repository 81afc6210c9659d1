"""Calls of linear attention that are refused before any launch, beside those of test_linattn_abi.  No
GPU needed."""
import ctypes

import pytest

import state_space_sequence_cumsum_amd as ssd
from state_space_sequence_cumsum_amd import linattn


def _problem(**kw):
    base = dict(batch=2, seqlen=100, nheads=8, ngroups=4, key_dim=64, value_dim=128, q_pitch=0,
                k_pitch=0, v_pitch=0, g_pitch=0, do_pitch=0, scale=1.0, decay=2, dtype=1)
    base.update(kw)
    return ssd.LinattnProblem(**base)


def _far(n):
    return [ctypes.c_void_p((i + 1) << 40) for i in range(n)]


@pytest.mark.parametrize("kw,fits", [
    (dict(nheads=16384, ngroups=1, key_dim=256), True),
    (dict(nheads=16384, ngroups=2, key_dim=256, decay=0), True),
    (dict(nheads=16385, ngroups=1, key_dim=256), False),
    (dict(nheads=16385, ngroups=1, key_dim=256, decay=0), False),
    (dict(nheads=40000, ngroups=1, key_dim=256), False),
    (dict(nheads=40000, ngroups=1, key_dim=256, decay=1), False),
    (dict(nheads=65535, ngroups=3, key_dim=72, dtype=0), False),
])
def test_gradient_rows_of_all_heads(kw, fits):
    """Every head's gradient of a shared q and k is a row of nheads * key_dim: the gradients bound
    it, the prompts, which have no such row, do not."""
    L, p = linattn.lib(), _problem(batch=1, seqlen=64, value_dim=8, **kw)
    assert L.ssd_linattn_validate(ctypes.byref(p)) == 0 and ssd.ssd_linattn_workspace_bytes(p) > 0
    assert (ssd.ssd_linattn_backward_workspace_bytes(p) > 0) == fits
    if not fits:
        a = _far(14)
        if p.decay != 2:
            a[11] = None
        assert L.ssd_linattn_backward(ctypes.byref(p), *a, 1 << 50, None) == 3


@pytest.mark.parametrize("kw", [
    dict(seqlen=100), dict(seqlen=128), dict(seqlen=128, nheads=16, value_dim=64), dict(seqlen=64, dtype=0),
    dict(seqlen=144, key_dim=72), dict(seqlen=72, key_dim=72, dtype=0)])
def test_only_the_final_state_may_be_the_initial_one(kw):
    """Also where o is as large as the states (bf16: 128 tokens with keys of 64)."""
    L, p = linattn.lib(), _problem(**kw)
    # q, k, v, g, h0, lengths, o, hT, workspace
    a = _far(9)
    a[6] = a[4]
    assert L.ssd_linattn(ctypes.byref(p), *a, 1 << 40, None) == 9
