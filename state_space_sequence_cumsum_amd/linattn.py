"""Linear attention with a decay for each head, and rotary positions for its queries and keys.

Argument marshalling only, as in :mod:`.block`, whose conventions hold: inputs may be column
slices of a wider projection output, outputs and states are contiguous and allocated when not given,
and every function calls the C entry point of the same name on the current (or given) HIP
stream.  Nothing here records a gradient: :func:`ssd_linattn_backward` and the inverse rotation
are calls of their own.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch import Tensor

from . import block
from .block import NO_WORKSPACE, _Bound, _call, _dense, _empty, _io, _rows, _stream

DECAY_NONE, DECAY_HEAD, DECAY_TOKEN = 0, 1, 2
POSITIONS_START, POSITIONS_FIRST, POSITIONS_EACH = 0, 1, 2


class LinattnProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seqlen", "nheads", "ngroups", "key_dim", "value_dim", "q_pitch", "k_pitch",
        "v_pitch", "g_pitch", "do_pitch")] + [
        ("scale", ctypes.c_float), ("decay", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class RotaryProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seqlen", "q_heads", "k_heads", "head_dim", "rotated", "q_pitch", "k_pitch")] + [
        ("scale", ctypes.c_float), ("positions", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("inverse", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_lib = None


def lib():
    """libssd.so with the argument types of this module's entry points."""
    global _lib
    if _lib is None:
        L = block.lib()
        vp, st, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        ap, rp = ctypes.POINTER(LinattnProblem), ctypes.POINTER(RotaryProblem)
        L.ssd_linattn_validate.argtypes, L.ssd_linattn_validate.restype = [ap], st
        L.ssd_linattn_workspace_bytes.argtypes, L.ssd_linattn_workspace_bytes.restype = [ap], sz
        L.ssd_linattn.argtypes, L.ssd_linattn.restype = [ap] + [vp] * 9 + [sz, vp], st
        L.ssd_linattn_step.argtypes, L.ssd_linattn_step.restype = [ap] + [vp] * 7, st
        L.ssd_linattn_backward_workspace_bytes.argtypes = [ap]
        L.ssd_linattn_backward_workspace_bytes.restype = sz
        L.ssd_linattn_backward.argtypes, L.ssd_linattn_backward.restype = [ap] + [vp] * 14 + [sz, vp], st
        L.ssd_rotary_validate.argtypes, L.ssd_rotary_validate.restype = [rp], st
        L.ssd_rotary.argtypes, L.ssd_rotary.restype = [rp] + [vp] * 7, st
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def _inputs(q, k, v, g, scale, lead):
    """(problem, GPU, addresses of q, k, v, g)."""
    code, dev = _io(q, "q")
    td = q.dtype
    if not (isinstance(v, Tensor) and q.dim() == lead + 2 and v.dim() == lead + 2):
        names = "[b, L, groups, key]" if lead == 2 else "[b, groups, key]"
        raise ValueError(f"linear attention takes q and k {names}, and v with [heads, value] in "
                         "place of the last two")
    tokens, (G, dk), (H, dv) = q.shape[:lead], q.shape[lead:], v.shape[lead:]
    qp, q_pitch = _rows(q, "q", td, q.shape, dev, lead)
    kp, k_pitch = _rows(k, "k", td, q.shape, dev, lead)
    vp, v_pitch = _rows(v, "v", td, (*tokens, H, dv), dev, lead)
    gp, g_pitch, decay = None, 0, DECAY_NONE
    if g is not None:
        if isinstance(g, Tensor) and g.dim() == 1:
            gp, decay = _dense(g, "g", torch.float32, (H,), dev), DECAY_HEAD
        else:
            (gp, g_pitch), decay = _rows(g, "g", td, (*tokens, H), dev, lead), DECAY_TOKEN
    b, L = tokens[0], tokens[1] if lead == 2 else 1
    prob = LinattnProblem(b, L, H, G, dk, dv, q_pitch, k_pitch, v_pitch, g_pitch, 0, scale, decay,
                          code)
    return prob, dev, (qp, kp, vp, gp)


def linattn_problem(q, v, *, decay=DECAY_TOKEN, scale=1.0) -> LinattnProblem:
    """The problem of linear attention over dense q [b, L, groups, key] and v [b, L, heads, value]."""
    return LinattnProblem(*q.shape[:2], v.shape[2], *q.shape[2:], v.shape[3], 0, 0, 0, 0, 0, scale,
                          decay, _io(q, "q")[0])


def ssd_linattn_workspace_bytes(problem: LinattnProblem) -> int:
    """Bytes of workspace ssd_linattn needs (1: none); 0 when the problem is not valid."""
    return lib().ssd_linattn_workspace_bytes(ctypes.byref(problem))


def ssd_linattn_backward_workspace_bytes(problem: LinattnProblem) -> int:
    """Bytes of workspace ssd_linattn_backward needs (1: none); 0 when it does not take the problem."""
    return lib().ssd_linattn_backward_workspace_bytes(ctypes.byref(problem))


def _workspace(workspace, need, dev, device, stream):
    """(workspace tensor or None, its address, its bytes) for `need` bytes; 0: the call is refused."""
    if workspace is not None:
        if not (isinstance(workspace, Tensor) and workspace.get_device() == dev
                and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need <= NO_WORKSPACE:
        return None, None, need
    workspace = _empty(need, torch.uint8, device, stream)
    return workspace, workspace.data_ptr(), need


def ssd_linattn(q, k, v, g=None, h0=None, *, scale=1.0, lengths=None, o=None, hT=None,
                want_final=True, workspace=None, stream=None):
    """Linear attention over prompts: S_t = exp(g_t) S_(t-1) + v_t k_t^T, o_t = scale S_t q_t.

    q, k [b, L, groups, key] and v [b, L, heads, value] (float32 or bfloat16; may be column
    slices whose rows start on 16 bytes; heads a multiple of groups, head h reads group
    h // (heads // groups)); ``g`` the log decays: [b, L, heads] in the same type, [heads]
    float32 (the same for every token), or None (no decay); values above 0 are taken as 0.  h0
    [b, heads, value, key] float32 (None: zeros).  ``lengths`` [b] int32: tokens of each
    sequence; rows behind them are left as they were in a given o and zeros in one allocated
    here, and hT is the state after each sequence's own last token.  hT may be h0 itself.
    Returns (o [b, L, heads, value], hT or None)."""
    prob, dev, ptrs = _inputs(q, k, v, g, scale, 2)
    td, device = q.dtype, q.device
    states = (prob.batch, prob.nheads, prob.value_dim, prob.key_dim)
    hp = _dense(h0, "h0", torch.float32, states, dev)
    lp = _dense(lengths, "lengths", torch.int32, (prob.batch,), dev)
    if o is None:
        o = _empty(v.shape, td, device, stream, torch.empty if lengths is None else torch.zeros)
        op = o.data_ptr()
    else:
        op = _dense(o, "o", td, v.shape, dev)
    if hT is None and want_final:
        hT = _empty(states, torch.float32, device, stream)
        tp = hT.data_ptr()
    else:
        tp = _dense(hT, "hT", torch.float32, states, dev)
    L, p = lib(), ctypes.byref(prob)
    need = L.ssd_linattn_workspace_bytes(p) if workspace is None else 0
    workspace, wp, n = _workspace(workspace, need, dev, device, stream)
    _call(L.ssd_linattn, (p, *ptrs, hp, lp, op, tp, wp, n, _stream(stream, dev)), dev, "ssd_linattn")
    return o, hT


def ssd_linattn_backward(do, q, k, v, g=None, h0=None, dhT=None, *, scale=1.0, lengths=None, dq=None,
                         dk=None, dv=None, dg=None, dh0=None, want_dg=True, want_dh0=True,
                         workspace=None, stream=None):
    """Gradients of ssd_linattn's inputs from ``do`` [b, L, heads, value], that of its o (may be
    a column slice), and ``dhT``, that of its hT (None: zeros).  The other inputs are the forward
    call's; its outputs are not needed.  heads * key may be 2^22 at most.

    Returns (dq, dk, dv, dg, dh0), each of its input's shape and type: dg None without a per-token
    g (fixed decays have no gradient here) or with want_dg False, dh0 None without an h0 or
    with want_dh0 False.  In bfloat16 dq and dk have other last bits without dg.  Rows behind a
    sequence's length are left as they were in given outputs and zeros in those allocated here."""
    prob, dev, ptrs = _inputs(q, k, v, g, scale, 2)
    td, device = q.dtype, q.device
    dp, prob.do_pitch = _rows(do, "do", td, v.shape, dev, 2)
    states = (prob.batch, prob.nheads, prob.value_dim, prob.key_dim)
    hp = _dense(h0, "h0", torch.float32, states, dev)
    tp = _dense(dhT, "dhT", torch.float32, states, dev)
    lp = _dense(lengths, "lengths", torch.int32, (prob.batch,), dev)
    make = torch.empty if lengths is None else torch.zeros
    outs = []
    for t, name, shape, dtype, want in (
            (dq, "dq", q.shape, td, True), (dk, "dk", q.shape, td, True), (dv, "dv", v.shape, td, True),
            (dg, "dg", v.shape[:3], td, want_dg and prob.decay == DECAY_TOKEN),
            (dh0, "dh0", states, torch.float32, want_dh0 and h0 is not None)):
        if t is not None:
            _dense(t, name, dtype, shape, dev)
        elif want:
            t = _empty(shape, dtype, device, stream, make if name != "dh0" else torch.empty)
        outs.append(t)
    L, p = lib(), ctypes.byref(prob)
    need = L.ssd_linattn_backward_workspace_bytes(p) if workspace is None else 0
    workspace, wp, n = _workspace(workspace, need, dev, device, stream)
    _call(L.ssd_linattn_backward,
          (p, dp, *ptrs, hp, tp, lp, *[None if t is None else t.data_ptr() for t in outs], wp, n,
           _stream(stream, dev)), dev, "ssd_linattn_backward")
    return tuple(outs)


def _step_args(q, k, v, h, g, scale, o, stream):
    prob, dev, ptrs = _inputs(q, k, v, g, scale, 1)
    if h is None:
        raise ValueError("h must be a GPU tensor")
    hp = _dense(h, "h", torch.float32, (prob.batch, prob.nheads, prob.value_dim, prob.key_dim), dev)
    if o is None:
        o = _empty(v.shape, v.dtype, v.device, stream)
    op = _dense(o, "o", v.dtype, v.shape, dev)
    return (ctypes.byref(prob), *ptrs, hp, op, _stream(stream, dev)), dev, o


def ssd_linattn_step(q, k, v, h, g=None, *, scale=1.0, o=None, stream=None):
    """Linear attention for one token per sequence: q, k [b, groups, key], v [b, heads, value],
    g [b, heads], [heads] float32 or None; h [b, heads, value, key] float32 is updated in
    place.  Returns o [b, heads, value]."""
    args, dev, o = _step_args(q, k, v, h, g, scale, o, stream)
    _call(lib().ssd_linattn_step, args, dev, "ssd_linattn_step")
    return o


class LinattnStepPlan(_Bound):
    """ssd_linattn_step bound to fixed tensors, for decode loops: the arguments are checked
    once, and run() only calls the C entry point (the caller refills q, k, v and g in place; h
    is updated in place).  The stream is fixed when the plan is made."""

    def __init__(self, q, k, v, h, g=None, *, scale=1.0, o=None, stream=None):
        args, dev, o = _step_args(q, k, v, h, g, scale, o, stream)
        super().__init__(lib().ssd_linattn_step, args, dev, "ssd_linattn_step", (q, k, v, h, g), o)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rotary_frequencies(rotated, base=10000.0, *, scaling=None, factor=1.0, length=None, slow=1.0,
                       fast=32.0, device=None):
    """Radians per position of each pair, [rotated / 2] float32: base^(-2j / rotated), and for
    contexts ``factor`` times longer than the ``length`` tokens a model was trained with:

    * ``"linear"``: every frequency divided by factor (positions interpolated);
    * ``"base"``: the base grown so that the slowest pair turns factor times slower and the
      fastest ones keep their frequency;
    * ``"parts"``: pairs that turn more than ``fast`` times within ``length`` keep their
      frequency, those that turn less than ``slow`` times are divided by factor, and between
      them the two are mixed in proportion to the turns' place between ``slow`` and ``fast``.

    Computed in 64 bits on the host and rounded once."""
    if rotated <= 0 or rotated % 2:
        raise ValueError(f"rotated must be positive and even, not {rotated}")
    if not (factor > 0 and math.isfinite(factor) and base > 0 and math.isfinite(base)):
        raise ValueError("base and factor must be positive")
    j = torch.arange(0, rotated, 2, dtype=torch.float64)
    if scaling == "base":
        if rotated < 4:
            raise ValueError("a single pair has no slower one: scaling \"base\" takes rotated >= 4")
        base = base * factor ** (rotated / (rotated - 2))
    freqs = base ** (-j / rotated)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "parts":
        if length is None or not length > 0 or not 0 <= slow < fast:
            raise ValueError("scaling \"parts\" takes length > 0 and 0 <= slow < fast")
        turns = length * freqs / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freqs = freqs / factor * (1 - keep) + freqs * keep
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', not {scaling!r}")
    return freqs.float().to(device)


def ssd_rotary(q, k, freqs, positions=None, *, interleaved=False, inverse=False, scale=1.0,
               q_out=None, k_out=None, stream=None):
    """Rotary positions of queries and keys, in one launch.

    q [b, L, heads, width] and k [b, L, groups, width] or None (float32 or bfloat16; may be
    column slices), or one token per sequence: q [b, heads, width].  The first 2 * len(freqs)
    elements of every head are turned in pairs (j, j + len(freqs)), or (2j, 2j + 1) when
    ``interleaved``, by position * freqs[j] radians (``freqs`` float32,
    :func:`rotary_frequencies`), and multiplied by ``scale``; the others are copied.
    ``positions`` int32: [b], the position of each sequence's first token (single tokens: of the
    token); [b, L], of every token; None: from 0.  ``inverse`` turns back, as the gradient
    does.  Outputs may be q and k themselves where those are contiguous.  Returns q_out, or
    (q_out, k_out) with a k."""
    code, dev = _io(q, "q")
    td, shape = q.dtype, q.shape
    lead = len(shape) - 2
    if lead not in (1, 2):
        raise ValueError("ssd_rotary takes q [b, L, heads, width] or [b, heads, width]")
    b, hq, width = shape[0], shape[-2], shape[-1]
    L = shape[1] if lead == 2 else 1
    qp, q_pitch = _rows(q, "q", td, shape, dev, lead)
    kp, k_pitch, hk, k_shape = None, 0, 0, None
    if k is not None:
        if not isinstance(k, Tensor) or k.dim() != lead + 2:
            raise ValueError("k must be a GPU tensor with q's dimensions")
        hk = k.shape[lead]
        k_shape = (b, L, hk, width) if lead == 2 else (b, hk, width)
        kp, k_pitch = _rows(k, "k", td, k_shape, dev, lead)
        if hk == 0:
            raise ValueError("k has no heads: give None")
    elif k_out is not None:
        raise ValueError("k_out without a k")
    if not isinstance(freqs, Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be [rotated / 2]")
    fp = _dense(freqs, "freqs", torch.float32, freqs.shape, dev)
    pp, mode = None, POSITIONS_START
    if positions is not None:
        each = lead == 2 and isinstance(positions, Tensor) and positions.dim() == 2
        pp = _dense(positions, "positions", torch.int32, (b, L) if each else (b,), dev)
        mode = POSITIONS_EACH if each else POSITIONS_FIRST
    if q_out is None:
        q_out = _empty(shape, td, q.device, stream)
        oq = q_out.data_ptr()
    else:
        oq = _dense(q_out, "q_out", td, shape, dev)
    ok = None
    if k is not None:
        if k_out is None:
            k_out = _empty(k_shape, td, q.device, stream)
            ok = k_out.data_ptr()
        else:
            ok = _dense(k_out, "k_out", td, k_shape, dev)
    prob = RotaryProblem(b, L, hq, hk, width, 2 * freqs.shape[0], q_pitch, k_pitch, scale, mode,
                         1 if interleaved else 0, 1 if inverse else 0, code)
    _call(lib().ssd_rotary, (ctypes.byref(prob), qp, kp, fp, pp, oq, ok, _stream(stream, dev)), dev,
          "ssd_rotary")
    return q_out if k is None else (q_out, k_out)
