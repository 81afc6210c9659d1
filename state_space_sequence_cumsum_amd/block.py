"""The operators around the SSD forward: short causal convolution, selective scan, block norms.

Argument marshalling only, as in :mod:`.binding`: every function checks placement, dtype,
shape and layout of its tensors and calls the C entry point of the same name on the current
(or given) HIP stream.  Inputs may be column slices of a wider projection output (rows dense,
one pitch from token to token); outputs and states are contiguous and allocated with
``torch.empty`` when not given.  Forward only: none of these functions records a gradient.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import SSD_BF16, SSD_F32, _raise, _stream

_DTYPES = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


class ConvProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("x_pitch", ctypes.c_int64), ("split", ctypes.c_int64 * 3), ("width", ctypes.c_int32),
                ("silu", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class ScanProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seqlen", "channels", "ngroups", "dstate", "x_pitch", "dt_pitch", "z_pitch",
        "B_pitch", "C_pitch")] + [("softplus", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("x_pitch", ctypes.c_int64), ("z_pitch", ctypes.c_int64), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("gate_after", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32)]


_lib = None


def lib():
    """libssd.so with the argument types of this module's entry points."""
    global _lib
    if _lib is None:
        L = binding.lib()
        vp, st, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        cp, sp, np_ = (ctypes.POINTER(t) for t in (ConvProblem, ScanProblem, NormProblem))
        L.ssd_conv_validate.argtypes, L.ssd_conv_validate.restype = [cp], st
        L.ssd_conv.argtypes, L.ssd_conv.restype = [cp] + [vp] * 10, st
        L.ssd_conv_step.argtypes, L.ssd_conv_step.restype = [cp] + [vp] * 8, st
        L.ssd_scan_validate.argtypes, L.ssd_scan_validate.restype = [sp], st
        L.ssd_scan_workspace_bytes.argtypes, L.ssd_scan_workspace_bytes.restype = [sp], sz
        L.ssd_scan.argtypes, L.ssd_scan.restype = [sp] + [vp] * 13 + [sz, vp], st
        L.ssd_scan_step.argtypes, L.ssd_scan_step.restype = [sp] + [vp] * 11, st
        L.ssd_norm_validate.argtypes, L.ssd_norm_validate.restype = [np_], st
        L.ssd_norm.argtypes, L.ssd_norm.restype = [np_] + [vp] * 7, st
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# tensor checks
# ---------------------------------------------------------------------------
def _check(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dense(t, name, dtype, shape, device):
    """The address of a contiguous tensor (None for None)."""
    if t is None:
        return None
    _check(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, shape, device, lead):
    """(address, pitch) of a tensor whose first `lead` dimensions count tokens: the others
    are dense, and the tokens follow each other at one pitch."""
    _check(t, name, dtype, shape, device)
    stride, width = t.stride(), 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and stride[d] != width:
            raise ValueError(f"{name} must have dense rows")
        width *= shape[d]
    pitch, tokens = 0, 1
    for d in range(lead - 1, -1, -1):
        if shape[d] != 1:
            if pitch == 0:
                pitch = stride[d] // tokens
                if pitch < width:
                    raise ValueError(f"{name} has overlapping rows")
            if stride[d] != pitch * tokens:
                raise ValueError(f"{name} must have one pitch from token to token")
        tokens *= shape[d]
    return t.data_ptr(), pitch


def _io(x, name="x"):
    code = _DTYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if code is None:
        raise ValueError(f"{name} must be a float32 or bfloat16 GPU tensor")
    return code


class _Call:
    """A C entry point with checked arguments: what a plan keeps and a function calls once."""

    __slots__ = ("fn", "args", "device", "what", "keep")

    def __init__(self, fn, args, device, what, keep):
        self.fn, self.args, self.device, self.what, self.keep = fn, args, device, what, keep

    def __call__(self):
        # kernels are launched for the tensors' device, whichever is current
        if torch.cuda.current_device() == self.device.index:
            st = self.fn(*self.args)
        else:
            with torch.cuda.device(self.device):
                st = self.fn(*self.args)
        if st != 0:
            _raise(st, self.what)


# ---------------------------------------------------------------------------
# short causal convolution
# ---------------------------------------------------------------------------
def _conv_call(x, weight, bias, state, silu, lengths, split, y, final_state, want_final, stream,
               step):
    what = "ssd_conv_step" if step else "ssd_conv"
    code = _io(x)
    if x.dim() != (2 if step else 3):
        raise ValueError(f"{what} takes x " + ("[b, channels]" if step else "[b, L, channels]"))
    if weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    td, dev, lead = x.dtype, x.device, tuple(x.shape[:-1])
    b, c = x.shape[0], x.shape[-1]
    k = weight.shape[1]
    one = split is None
    widths = [c] if one else [int(w) for w in split]
    if not 1 <= len(widths) <= 3 or sum(widths) != c or min(widths) <= 0:
        raise ValueError(f"split {widths} must be 1 to 3 positive widths with sum {c}")
    xp, pitch = _rows(x, "x", td, x.shape, None, len(lead))
    wp = _dense(weight, "weight", torch.float32, (c, k), dev)
    bp = _dense(bias, "bias", torch.float32, (c,), dev)
    sp = _dense(state, "state", td, (b, k - 1, c), dev)
    if y is None:
        ys = [torch.empty(*lead, w, device=dev, dtype=td) for w in widths]
    else:
        ys = [y] if isinstance(y, torch.Tensor) else list(y)
    if len(ys) != len(widths):
        raise ValueError(f"y must be {len(widths)} tensors, one per split width")
    yp = [_dense(t, "y", td, (*lead, w), dev) for t, w in zip(ys, widths)]
    yp += [None] * (3 - len(yp))
    prob = ConvProblem(b, 1 if step else x.shape[1], c, pitch,
                       (ctypes.c_int64 * 3)(*widths, *[0] * (3 - len(widths))), k, int(bool(silu)),
                       code)
    out = ys[0] if one else tuple(ys)
    if step:
        if state is None:
            raise ValueError("state must be a GPU tensor")
        args = (ctypes.byref(prob), xp, wp, bp, sp, *yp, _stream(stream, dev))
        call = _Call(lib().ssd_conv_step, args, dev, what, (prob, x, weight, bias, state, ys))
        return call, out, state
    lp = _dense(lengths, "lengths", torch.int32, (b,), dev)
    if final_state is None and want_final:
        final_state = torch.empty(b, k - 1, c, device=dev, dtype=td)
    fp = _dense(final_state, "final_state", td, (b, k - 1, c), dev)
    args = (ctypes.byref(prob), xp, wp, bp, sp, lp, *yp, fp, _stream(stream, dev))
    call = _Call(lib().ssd_conv, args, dev, what, (prob, x, weight, bias, state, lengths, ys,
                                                   final_state))
    return call, out, final_state


def ssd_conv(x, weight, bias=None, state=None, *, silu=True, lengths=None, split=None, y=None,
             final_state=None, want_final=True, stream=None):
    """Short causal depthwise convolution over prompts.

    x [b, L, channels] (float32 or bfloat16; may be a column slice); weight [channels, width]
    with 2 to 4 taps and bias [channels], float32; state [b, width-1, channels] the inputs
    before the first token (None: zeros).  ``split``: up to three widths with sum channels,
    the output then comes as that many contiguous tensors (x, B and C of ssd_forward).
    ``lengths`` [b] int32: tokens of each sequence; rows of y behind them are left as they
    were.  ``final_state`` may be ``state`` itself.  Returns (y or a tuple of them, final
    state or None)."""
    call, out, final = _conv_call(x, weight, bias, state, silu, lengths, split, y, final_state,
                                  want_final, stream, False)
    call()
    return out, final


def ssd_conv_step(x, weight, bias, state, *, silu=True, split=None, y=None, stream=None):
    """The convolution for one token per sequence: x [b, channels]; state [b, width-1,
    channels] is shifted in place.  Returns y, or a tuple of them where ``split`` is given."""
    call, out, _ = _conv_call(x, weight, bias, state, silu, None, split, y, None, False, stream,
                              True)
    call()
    return out


class ConvStepPlan:
    """ssd_conv_step bound to fixed tensors, for decode loops: the arguments are checked
    once, and run() only calls the C entry point (the caller refills x in place; state is
    updated in place).  The stream is fixed when the plan is made."""

    def __init__(self, x, weight, bias, state, *, silu=True, split=None, y=None, stream=None):
        self._call, self.y, _ = _conv_call(x, weight, bias, state, silu, None, split, y, None,
                                           False, stream, True)

    def run(self):
        """One step; returns y (the same tensors every call)."""
        self._call()
        return self.y


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
def _scan_problem(x, dt, A, B, C, z, dt_softplus, lead):
    code = _io(x)
    if x.dim() != lead + 1 or B.dim() != lead + 2 or A.dim() != 2:
        names = "[b, L, channels]" if lead == 2 else "[b, channels]"
        raise ValueError(f"the scan takes x {names}, B with [ngroups, dstate] in place of "
                         "channels, and A [channels, dstate]")
    td, dev = x.dtype, x.device
    c, (G, N) = x.shape[-1], B.shape[-2:]
    xp, x_pitch = _rows(x, "x", td, x.shape, None, lead)
    dp, dt_pitch = _rows(dt, "dt", td, x.shape, dev, lead)
    ap = _dense(A, "A", torch.float32, (c, N), dev)
    bc = (*x.shape[:-1], G, N)
    bp, b_pitch = _rows(B, "B", td, bc, dev, lead)
    cp, c_pitch = _rows(C, "C", td, bc, dev, lead)
    zp, z_pitch = (None, 0) if z is None else _rows(z, "z", td, x.shape, dev, lead)
    prob = ScanProblem(x.shape[0], x.shape[1] if lead == 2 else 1, c, G, N, x_pitch, dt_pitch,
                       z_pitch, b_pitch, c_pitch, int(bool(dt_softplus)), code)
    return prob, td, dev, (xp, dp, ap, bp, cp), zp


def scan_problem(x, B, *, dt_softplus=False) -> ScanProblem:
    """The problem of a scan over dense x [b, L, channels] and B [b, L, ngroups, dstate]."""
    return ScanProblem(x.shape[0], x.shape[1], x.shape[2], B.shape[2], B.shape[3], 0, 0, 0, 0, 0,
                       int(bool(dt_softplus)), _io(x))


def ssd_scan_workspace_bytes(problem: ScanProblem) -> int:
    """Bytes of workspace ssd_scan needs; 0 when the problem is not valid."""
    return lib().ssd_scan_workspace_bytes(ctypes.byref(problem))


def ssd_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, dt_softplus=False,
             lengths=None, y=None, hT=None, want_final=True, workspace=None, stream=None):
    """Selective scan over prompts, with a decay rate per channel and state.

    x, dt and z (the gate, optional) [b, L, channels]; B, C [b, L, ngroups, dstate]; A
    [channels, dstate], D and dt_bias [channels] (optional) and h0 [b, channels, dstate]
    (None: zeros) float32.  ``dt_softplus``: the step size is log(1 + exp(dt + dt_bias)).
    ``lengths`` [b] int32: tokens of each sequence; rows of y behind them are left as they
    were and hT is the state after each sequence's own last token.  hT may be h0 itself.
    Returns (y [b, L, channels], hT [b, channels, dstate] float32 or None)."""
    prob, td, dev, ptrs, zp = _scan_problem(x, dt, A, B, C, z, dt_softplus, 2)
    b, c, N = prob.batch, prob.channels, prob.dstate
    vec = [_dense(t, n, torch.float32, (c,), dev) for t, n in ((D, "D"), (dt_bias, "dt_bias"))]
    hp = _dense(h0, "h0", torch.float32, (b, c, N), dev)
    lp = _dense(lengths, "lengths", torch.int32, (b,), dev)
    if y is None:
        y = torch.empty(x.shape, device=dev, dtype=td)
    yp = _dense(y, "y", td, x.shape, dev)
    if hT is None and want_final:
        hT = torch.empty(b, c, N, device=dev, dtype=torch.float32)
    tp = _dense(hT, "hT", torch.float32, (b, c, N), dev)
    L = lib()
    if workspace is None:
        n = L.ssd_scan_workspace_bytes(ctypes.byref(prob))
        if n == 0:
            _raise(L.ssd_scan_validate(ctypes.byref(prob)), "ssd_scan")
        workspace = torch.empty(n, device=dev, dtype=torch.uint8)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    _Call(L.ssd_scan, (ctypes.byref(prob), *ptrs, vec[0], zp, vec[1], hp, lp, yp, tp,
                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                       _stream(stream, dev)), dev, "ssd_scan", None)()
    return y, hT


def _scan_step_call(x, dt, A, B, C, h, D, z, dt_bias, dt_softplus, y, stream):
    prob, td, dev, ptrs, zp = _scan_problem(x, dt, A, B, C, z, dt_softplus, 1)
    c, N = prob.channels, prob.dstate
    vec = [_dense(t, n, torch.float32, (c,), dev) for t, n in ((D, "D"), (dt_bias, "dt_bias"))]
    if h is None:
        raise ValueError("h must be a GPU tensor")
    hp = _dense(h, "h", torch.float32, (prob.batch, c, N), dev)
    if y is None:
        y = torch.empty(x.shape, device=dev, dtype=td)
    yp = _dense(y, "y", td, x.shape, dev)
    args = (ctypes.byref(prob), *ptrs, vec[0], zp, vec[1], hp, yp, _stream(stream, dev))
    return _Call(lib().ssd_scan_step, args, dev, "ssd_scan_step",
                 (prob, x, dt, A, B, C, h, D, z, dt_bias, y)), y


def ssd_scan_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, dt_softplus=False, y=None,
                  stream=None):
    """The scan for one token per sequence: x, dt, z [b, channels], B and C [b, ngroups,
    dstate]; h [b, channels, dstate] float32 is updated in place.  Returns y [b, channels]."""
    call, y = _scan_step_call(x, dt, A, B, C, h, D, z, dt_bias, dt_softplus, y, stream)
    call()
    return y


class ScanStepPlan:
    """ssd_scan_step bound to fixed tensors, for decode loops: the arguments are checked
    once, and run() only calls the C entry point (the caller refills x, dt, B, C and z in
    place; h is updated in place).  The stream is fixed when the plan is made."""

    def __init__(self, x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, dt_softplus=False,
                 y=None, stream=None):
        self._call, self.y = _scan_step_call(x, dt, A, B, C, h, D, z, dt_bias, dt_softplus, y,
                                             stream)

    def run(self):
        """One step; returns y (the same tensor every call)."""
        self._call()
        return self.y


# ---------------------------------------------------------------------------
# block norms
# ---------------------------------------------------------------------------
def ssd_norm(x, weight, z=None, residual=None, *, ngroups=1, eps=1e-5, scale=1.0,
             gate_after=False, y=None, residual_out=None, want_residual=True, stream=None):
    """RMS norm before or after a block, with its gate and residual addition.

    x and z (the gate, optional) [..., channels]; weight [channels] float32; the mean square
    is taken over each of ``ngroups`` runs of channels.  The gate silu(z) multiplies x before
    the norm, or its result with ``gate_after``.  With ``residual`` [..., channels] (float32
    or x's dtype) the norm takes residual + scale * x (the gate applied), which is also
    stored to ``residual_out`` (may be ``residual`` itself).  Returns y, or (y,
    residual_out) with a residual (None in its place unless ``want_residual``)."""
    code = _io(x)
    if x.dim() < 1:
        raise ValueError("ssd_norm takes x [..., channels]")
    td, dev, c = x.dtype, x.device, x.shape[-1]
    lead = x.dim() - 1
    xp, x_pitch = _rows(x, "x", td, x.shape, None, lead)
    zp, z_pitch = (None, 0) if z is None else _rows(z, "z", td, x.shape, dev, lead)
    wp = _dense(weight, "weight", torch.float32, (c,), dev)
    rp = op = None
    rcode = SSD_F32
    if residual is not None:
        if residual.dtype not in (torch.float32, td):
            raise ValueError(f"residual has dtype {residual.dtype}, expected float32 or {td}")
        rcode = _DTYPES[residual.dtype]
        rp = _dense(residual, "residual", residual.dtype, x.shape, dev)
        if residual_out is None and want_residual:
            residual_out = torch.empty(x.shape, device=dev, dtype=residual.dtype)
        op = _dense(residual_out, "residual_out", residual.dtype, x.shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if y is None:
        y = torch.empty(x.shape, device=dev, dtype=td)
    yp = _dense(y, "y", td, x.shape, dev)
    rows = x.numel() // c if c else 0
    prob = NormProblem(rows, c, ngroups, x_pitch, z_pitch, eps, scale, int(bool(gate_after)), code,
                       rcode)
    _Call(lib().ssd_norm, (ctypes.byref(prob), xp, zp, rp, wp, yp, op, _stream(stream, dev)), dev,
          "ssd_norm", None)()
    return y if residual is None else (y, residual_out)
