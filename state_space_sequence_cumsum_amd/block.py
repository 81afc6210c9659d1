"""The operators around the SSD forward: short causal convolution, selective scan, block norms.

Argument marshalling only, as in :mod:`.binding`: every function checks placement, dtype,
shape and layout of its tensors and calls the C entry point of the same name on the current
(or given) HIP stream.  Inputs may be column slices of a wider projection output (rows dense,
one pitch from token to token); outputs and states are contiguous and allocated when not given
(with ``torch.empty``, or as zeros where ``lengths`` leave rows of them unwritten).  An output
may be a final state in its initial state's tensor, and in the step functions and the norm an
input of its own dense layout; otherwise one that shares memory with another argument is
refused.  Forward only: none of these functions records a gradient.
"""
from __future__ import annotations

import ctypes

import torch
from torch import Tensor

from . import binding
from .binding import SSD_BF16, SSD_F32, _raise

NO_WORKSPACE = 1    # SSD_SCAN_NO_WORKSPACE: a scan that needs up to this many bytes needs none
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
_one_gpu = False     # set with _lib: a single GPU is always the current one


def lib():
    """libssd.so with the argument types of this module's entry points."""
    global _lib, _one_gpu
    if _lib is None:
        # (the count is final once the GPUs are in use)
        _one_gpu = torch.cuda.is_initialized() and torch.cuda.device_count() == 1
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
# tensor checks: one test of everything first, the reason for a refusal only where it fails
# (these run for every tensor of every call)
# ---------------------------------------------------------------------------
def _refuse(t, name, dtype, shape, device):
    if not isinstance(t, Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dense(t, name, dtype, shape, device):
    """The address of a contiguous tensor on GPU `device` (None for None)."""
    if t is None:
        return None
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == device and t.is_contiguous()):
        _refuse(t, name, dtype, shape, device)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _pitch(t, name, lead):
    """Elements between the tokens of a tensor whose first `lead` dimensions count tokens: the
    others are dense, and the tokens follow each other at one pitch (0: dense tokens)."""
    shape, stride, width = t.shape, t.stride(), 1
    if lead == 2 and len(shape) == 3 and shape[1] > 1:      # the usual slice, without the loops
        b, L, c = shape
        pitch = stride[1]
        if pitch >= c and (c == 1 or stride[2] == 1) and (b == 1 or stride[0] == L * pitch):
            return pitch
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
    return pitch


def _rows(t, name, dtype, shape, device, lead):
    """(address, pitch) of a tensor on GPU `device` that _pitch takes."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == device):
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr(), 0 if t.is_contiguous() else _pitch(t, name, lead)


def _io(x, name="x"):
    """(dtype code, GPU index) of the tensor that sets both."""
    code = _DTYPES.get(x.dtype) if isinstance(x, Tensor) and x.is_cuda else None
    if code is None:
        raise ValueError(f"{name} must be a float32 or bfloat16 GPU tensor")
    return code, x.get_device()


def _empty(shape, dtype, device, stream, make=torch.empty):
    """A new tensor for a call on `stream` (None: the current one): it comes from that stream's
    memory, which earlier work on the current stream may not be using any more."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _cleared(lead, widths, dtype, device, stream):
    """New tensors [*lead, width] of zeros, for outputs whose rows behind a sequence's length the
    kernels leave as they are: parts of one buffer, each on 256 bytes, cleared by one launch."""
    if len(widths) == 1:
        return (_empty((*lead, widths[0]), dtype, device, stream, torch.zeros),)
    rows = lead[0] * lead[1]
    starts = [0]
    for w in widths:
        starts.append(starts[-1] + (rows * w + 127) // 128 * 128)
    whole = _empty((starts[-1],), dtype, device, stream, torch.zeros)
    return tuple([whole[at:at + rows * w].view(*lead, w) for at, w in zip(starts, widths)])


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(fn, args, device, what):
    """Calls a C entry point: kernels are launched for the tensors' GPU, whichever is current."""
    if _one_gpu or torch.cuda.current_device() == device:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != 0:
        _raise(st, what)


class _Bound:
    """A C entry point bound to fixed tensors (kept alive here); run() only calls it."""

    def __init__(self, fn, args, device, what, keep, y):
        self._fn, self._args, self._device, self._what = fn, args, device, what
        self._keep, self.y = keep, y

    def run(self):
        """One step; returns y (the same tensors every call)."""
        _call(self._fn, self._args, self._device, self._what)
        return self.y


# ---------------------------------------------------------------------------
# short causal convolution
# ---------------------------------------------------------------------------
def _conv_args(x, weight, bias, state, silu, lengths, split, y, final_state, want_final, stream,
               step):
    """(arguments of the entry point, GPU, outputs, final state, tensors to keep)."""
    what = "ssd_conv_step" if step else "ssd_conv"
    code, dev = _io(x)
    shape, td = x.shape, x.dtype
    if len(shape) != (2 if step else 3):
        raise ValueError(f"{what} takes x " + ("[b, channels]" if step else "[b, L, channels]"))
    if not isinstance(weight, Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    b, c, k = shape[0], shape[-1], weight.shape[1]
    lead = tuple(shape[:-1])
    widths = (c,) if split is None else tuple([int(w) for w in split])
    n = len(widths)
    if not 1 <= n <= 3 or sum(widths) != c or min(widths) <= 0:
        raise ValueError(f"split {list(widths)} must be 1 to 3 positive widths with sum {c}")
    xp, pitch = _rows(x, "x", td, shape, dev, len(lead))
    wp = _dense(weight, "weight", torch.float32, (c, k), dev)
    bp = _dense(bias, "bias", torch.float32, (c,), dev)
    sp = _dense(state, "state", td, (b, k - 1, c), dev)
    if y is None:
        if lengths is None:
            ys = tuple([_empty((*lead, w), td, x.device, stream) for w in widths])
        else:
            ys = _cleared(lead, widths, td, x.device, stream)
        yp = [t.data_ptr() for t in ys]
    else:
        ys = (y,) if isinstance(y, Tensor) else tuple(y)
        if len(ys) != n:
            raise ValueError(f"y must be {n} tensors, one per split width")
        yp = [_dense(t, "y", td, (*lead, w), dev) for t, w in zip(ys, widths)]
        if None in yp:
            raise ValueError("y must be a GPU tensor")
    yp += [None] * (3 - n)
    prob = ConvProblem(b, 1 if step else shape[1], c, pitch, widths, k, 1 if silu else 0, code)
    out = ys[0] if split is None else ys
    if step:
        if state is None:
            raise ValueError("state must be a GPU tensor")
        args = (ctypes.byref(prob), xp, wp, bp, sp, *yp, _stream(stream, dev))
        return args, dev, out, state, (x, weight, bias, state, ys)
    lp = _dense(lengths, "lengths", torch.int32, (b,), dev)
    if final_state is None and want_final:
        final_state = _empty((b, k - 1, c), td, x.device, stream)
        fp = final_state.data_ptr()
    else:
        fp = _dense(final_state, "final_state", td, (b, k - 1, c), dev)
    args = (ctypes.byref(prob), xp, wp, bp, sp, lp, *yp, fp, _stream(stream, dev))
    return args, dev, out, final_state, None


def ssd_conv(x, weight, bias=None, state=None, *, silu=True, lengths=None, split=None, y=None,
             final_state=None, want_final=True, stream=None):
    """Short causal depthwise convolution over prompts.

    x [b, L, channels] (float32 or bfloat16; may be a column slice); weight [channels, width]
    with 2 to 4 taps and bias [channels], float32; state [b, width-1, channels] the inputs
    before the first token (None: zeros).  ``split``: up to three widths with sum channels,
    the output then comes as that many contiguous tensors (x, B and C of ssd_forward).
    ``lengths`` [b] int32: tokens of each sequence; rows behind them are left as they were in a
    given y, and zeros in one allocated here (ssd_forward, which has no lengths, then takes x, B
    and C with a dt of zero behind them).  ``final_state`` may be ``state`` itself.  Returns (y or a tuple of them, final
    state or None)."""
    args, dev, out, final, _ = _conv_args(x, weight, bias, state, silu, lengths, split, y,
                                          final_state, want_final, stream, False)
    _call(lib().ssd_conv, args, dev, "ssd_conv")
    return out, final


def ssd_conv_step(x, weight, bias, state, *, silu=True, split=None, y=None, stream=None):
    """The convolution for one token per sequence: x [b, channels]; state [b, width-1,
    channels] is shifted in place.  Returns y, or a tuple of them where ``split`` is given."""
    args, dev, out, _, _ = _conv_args(x, weight, bias, state, silu, None, split, y, None, False,
                                      stream, True)
    _call(lib().ssd_conv_step, args, dev, "ssd_conv_step")
    return out


class ConvStepPlan(_Bound):
    """ssd_conv_step bound to fixed tensors, for decode loops: the arguments are checked
    once, and run() only calls the C entry point (the caller refills x in place; state is
    updated in place).  The stream is fixed when the plan is made."""

    def __init__(self, x, weight, bias, state, *, silu=True, split=None, y=None, stream=None):
        args, dev, out, _, keep = _conv_args(x, weight, bias, state, silu, None, split, y, None,
                                             False, stream, True)
        super().__init__(lib().ssd_conv_step, args, dev, "ssd_conv_step", keep, out)


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dt_softplus, lead):
    """(problem, GPU, addresses of x, dt, A, B, C, D, z, dt_bias)."""
    code, dev = _io(x)
    shape, td, f32 = x.shape, x.dtype, torch.float32
    if not (isinstance(A, Tensor) and isinstance(B, Tensor) and len(shape) == lead + 1
            and B.dim() == lead + 2 and A.dim() == 2):
        names = "[b, L, channels]" if lead == 2 else "[b, channels]"
        raise ValueError(f"the scan takes x {names}, B with [ngroups, dstate] in place of "
                         "channels, and A [channels, dstate]")
    b, L, c = shape[0], shape[1] if lead == 2 else 1, shape[-1]
    G, N = B.shape[-2:]
    bc = (b, L, G, N) if lead == 2 else (b, G, N)
    xp, x_pitch = _rows(x, "x", td, shape, dev, lead)
    dp, dt_pitch = _rows(dt, "dt", td, shape, dev, lead)
    ap = _dense(A, "A", f32, (c, N), dev)
    bp, b_pitch = _rows(B, "B", td, bc, dev, lead)
    cp, c_pitch = _rows(C, "C", td, bc, dev, lead)
    Dp = _dense(D, "D", f32, (c,), dev)
    zp, z_pitch = (None, 0) if z is None else _rows(z, "z", td, shape, dev, lead)
    tp = _dense(dt_bias, "dt_bias", f32, (c,), dev)
    prob = ScanProblem(b, L, c, G, N, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch,
                       1 if dt_softplus else 0, code)
    return prob, dev, (xp, dp, ap, bp, cp, Dp, zp, tp)


def scan_problem(x, B, *, dt_softplus=False) -> ScanProblem:
    """The problem of a scan over dense x [b, L, channels] and B [b, L, ngroups, dstate]."""
    return ScanProblem(*x.shape, *B.shape[2:], 0, 0, 0, 0, 0, int(bool(dt_softplus)), _io(x)[0])


def ssd_scan_workspace_bytes(problem: ScanProblem) -> int:
    """Bytes of workspace ssd_scan needs (1: none); 0 when the problem is not valid."""
    return lib().ssd_scan_workspace_bytes(ctypes.byref(problem))


def ssd_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, dt_softplus=False,
             lengths=None, y=None, hT=None, want_final=True, workspace=None, stream=None):
    """Selective scan over prompts, with a decay rate per channel and state.

    x, dt and z (the gate, optional) [b, L, channels]; B, C [b, L, ngroups, dstate]; A
    [channels, dstate], D and dt_bias [channels] (optional) and h0 [b, channels, dstate]
    (None: zeros) float32.  ``dt_softplus``: the step size is log(1 + exp(dt + dt_bias)).
    ``lengths`` [b] int32: tokens of each sequence; rows behind them are left as they were in a
    given y and zeros in one allocated here, and hT is the state after each sequence's own last token.  hT may be h0 itself.
    Returns (y [b, L, channels], hT [b, channels, dstate] float32 or None)."""
    prob, dev, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dt_softplus, 2)
    td, f32 = x.dtype, torch.float32
    states = (prob.batch, prob.channels, prob.dstate)
    hp = _dense(h0, "h0", f32, states, dev)
    lp = _dense(lengths, "lengths", torch.int32, (prob.batch,), dev)
    if y is None:
        y = _empty(x.shape, td, x.device, stream, torch.empty if lengths is None else torch.zeros)
        yp = y.data_ptr()
    else:
        yp = _dense(y, "y", td, x.shape, dev)
    if hT is None and want_final:
        hT = _empty(states, f32, x.device, stream)
        tp = hT.data_ptr()
    else:
        tp = _dense(hT, "hT", f32, states, dev)
    L, p = lib(), ctypes.byref(prob)
    if workspace is None:
        n = L.ssd_scan_workspace_bytes(p)
        if n == 0:
            _raise(L.ssd_scan_validate(p), "ssd_scan")
        if n > NO_WORKSPACE:
            workspace = _empty(n, torch.uint8, x.device, stream)
    else:
        if not (isinstance(workspace, Tensor) and workspace.get_device() == dev
                and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        n = workspace.numel() * workspace.element_size()
    _call(L.ssd_scan, (p, *ptrs, hp, lp, yp, tp, None if workspace is None else workspace.data_ptr(),
                       n, _stream(stream, dev)), dev, "ssd_scan")
    return y, hT


def _scan_step_args(x, dt, A, B, C, h, D, z, dt_bias, dt_softplus, y, stream):
    prob, dev, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dt_softplus, 1)
    if h is None:
        raise ValueError("h must be a GPU tensor")
    hp = _dense(h, "h", torch.float32, (prob.batch, prob.channels, prob.dstate), dev)
    if y is None:
        y = _empty(x.shape, x.dtype, x.device, stream)
    yp = _dense(y, "y", x.dtype, x.shape, dev)
    return (ctypes.byref(prob), *ptrs, hp, yp, _stream(stream, dev)), dev, y


def ssd_scan_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, dt_softplus=False, y=None,
                  stream=None):
    """The scan for one token per sequence: x, dt, z [b, channels], B and C [b, ngroups,
    dstate]; h [b, channels, dstate] float32 is updated in place.  Returns y [b, channels]."""
    args, dev, y = _scan_step_args(x, dt, A, B, C, h, D, z, dt_bias, dt_softplus, y, stream)
    _call(lib().ssd_scan_step, args, dev, "ssd_scan_step")
    return y


class ScanStepPlan(_Bound):
    """ssd_scan_step bound to fixed tensors, for decode loops: the arguments are checked
    once, and run() only calls the C entry point (the caller refills x, dt, B, C and z in
    place; h is updated in place).  The stream is fixed when the plan is made."""

    def __init__(self, x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, dt_softplus=False,
                 y=None, stream=None):
        args, dev, y = _scan_step_args(x, dt, A, B, C, h, D, z, dt_bias, dt_softplus, y, stream)
        super().__init__(lib().ssd_scan_step, args, dev, "ssd_scan_step",
                         (x, dt, A, B, C, h, D, z, dt_bias), y)


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
    code, dev = _io(x)
    shape, td = x.shape, x.dtype
    if len(shape) < 1:
        raise ValueError("ssd_norm takes x [..., channels]")
    c, lead = shape[-1], len(shape) - 1
    xp, x_pitch = _rows(x, "x", td, shape, dev, lead)
    zp, z_pitch = (None, 0) if z is None else _rows(z, "z", td, shape, dev, lead)
    wp = _dense(weight, "weight", torch.float32, (c,), dev)
    rp = op = None
    rcode = SSD_F32
    if residual is not None:
        rd = residual.dtype if isinstance(residual, Tensor) else None
        if rd is not td and rd is not torch.float32:
            raise ValueError(f"residual has dtype {rd}, expected float32 or {td}")
        rcode = _DTYPES[rd]
        rp = _dense(residual, "residual", rd, shape, dev)
        if residual_out is None and want_residual:
            residual_out = _empty(shape, rd, x.device, stream)
            op = residual_out.data_ptr()
        else:
            op = _dense(residual_out, "residual_out", rd, shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if y is None:
        y = _empty(shape, td, x.device, stream)
        yp = y.data_ptr()
    else:
        yp = _dense(y, "y", td, shape, dev)
    prob = NormProblem(x.numel() // c if c else 0, c, ngroups, x_pitch, z_pitch, eps, scale,
                       1 if gate_after else 0, code, rcode)
    _call(lib().ssd_norm, (ctypes.byref(prob), xp, zp, rp, wp, yp, op, _stream(stream, dev)), dev,
          "ssd_norm")
    return y if residual is None else (y, residual_out)
