"""Bindings of the layer operators around the recurrence (``include/mamba3.h``, "Operators of the
layers" and "Operators of a gated recurrent layer"): the short causal convolution, the selective scan and
the residual RMS norm; the gated linear recurrence, the group norm and the cache of states in 8 or 4 bits.

As in the package's other bindings, every step of the computation runs in the library's HIP kernels;
this module checks shapes, types and devices, allocates outputs and workspaces where they are not
given, and passes the stream. Token arrays may be views of wider rows (their innermost dimensions
dense, one distance from token to token); every other tensor is contiguous. Calls run on the current
stream of x's device unless a stream of that device is given.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

from . import MAMBA3_BF16, MAMBA3_F32, MAMBA3_OK, Mamba3Error, lib

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_size = ctypes.c_size_t

MAMBA3_E4M3, MAMBA3_INT8 = 0, 1
MAMBA3_GATE_DECAY, MAMBA3_GATE_FORGET = 0, 1
MAMBA3_GN_NONE, MAMBA3_GN_SILU, MAMBA3_GN_GATE, MAMBA3_GN_PREGATE = range(4)
MAMBA3_CACHE_E4M3, MAMBA3_CACHE_INT8, MAMBA3_CACHE_INT4 = range(3)

_FORMS = {"decay": MAMBA3_GATE_DECAY, "forget": MAMBA3_GATE_FORGET}
_ACTS = {"none": MAMBA3_GN_NONE, "silu": MAMBA3_GN_SILU, "gate": MAMBA3_GN_GATE, "pregate": MAMBA3_GN_PREGATE}


@functools.lru_cache(None)
def _dtypes():
    import torch
    return {torch.bfloat16: MAMBA3_BF16, torch.float32: MAMBA3_F32}


@functools.lru_cache(None)
def _qtypes():
    import torch
    return {"e4m3": (MAMBA3_E4M3, torch.float8_e4m3fn), "int8": (MAMBA3_INT8, torch.int8)}


@functools.lru_cache(None)
def _kinds():
    import torch
    return {"e4m3": (MAMBA3_CACHE_E4M3, torch.float8_e4m3fn), "int8": (MAMBA3_CACHE_INT8, torch.int8),
            "int4": (MAMBA3_CACHE_INT4, torch.uint8)}


class ConvArgs(ctypes.Structure):
    """Mirror of ``mamba3_conv_args``."""
    _fields_ = [("batch", _i32), ("seqlen", _i32), ("dim", _i32), ("width", _i32), ("dtype", _i32), ("silu", _i32),
                ("cu_seqlens", _vp), ("nseq", _i32), ("x_row", _i64), ("x", _vp), ("weight", _vp), ("bias", _vp),
                ("conv_in", _vp), ("y", _vp), ("conv_out", _vp)]


class ConvBwdArgs(ctypes.Structure):
    """Mirror of ``mamba3_conv_bwd_args``."""
    _fields_ = [("fwd", ConvArgs), ("dy_row", _i64), ("dy", _vp), ("dconv_out", _vp), ("dx", _vp), ("dweight", _vp),
                ("dbias", _vp), ("dconv_in", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class ConvStepArgs(ctypes.Structure):
    """Mirror of ``mamba3_conv_step_args``."""
    _fields_ = [("batch", _i32), ("dim", _i32), ("width", _i32), ("dtype", _i32), ("silu", _i32), ("x_row", _i64),
                ("x", _vp), ("weight", _vp), ("bias", _vp), ("conv", _vp), ("y", _vp), ("slots", _vp),
                ("nslots", _i32)]


class SelectiveScanArgs(ctypes.Structure):
    """Mirror of ``mamba3_selective_scan_args``."""
    _fields_ = [("batch", _i32), ("seqlen", _i32), ("dim", _i32), ("dstate", _i32), ("ngroups", _i32),
                ("dtype", _i32), ("dt_softplus", _i32), ("cu_seqlens", _vp), ("nseq", _i32),
                ("x_row", _i64), ("dt_row", _i64), ("B_row", _i64), ("C_row", _i64), ("z_row", _i64),
                ("x", _vp), ("dt", _vp), ("B", _vp), ("C", _vp), ("z", _vp), ("A", _vp), ("D", _vp),
                ("dt_bias", _vp), ("h_in", _vp), ("y", _vp), ("h_out", _vp), ("workspace", _vp),
                ("workspace_bytes", _size)]


class SelectiveScanBwdArgs(ctypes.Structure):
    """Mirror of ``mamba3_selective_scan_bwd_args``."""
    _fields_ = [("fwd", SelectiveScanArgs), ("dy_row", _i64), ("dy", _vp), ("dh_out", _vp), ("dx", _vp), ("ddt", _vp),
                ("dB", _vp), ("dC", _vp), ("dz", _vp), ("dA", _vp), ("dD", _vp), ("ddt_bias", _vp), ("dh_in", _vp),
                ("workspace", _vp), ("workspace_bytes", _size)]


class SelectiveStepArgs(ctypes.Structure):
    """Mirror of ``mamba3_selective_step_args``."""
    _fields_ = [("batch", _i32), ("dim", _i32), ("dstate", _i32), ("ngroups", _i32), ("dtype", _i32),
                ("dt_softplus", _i32), ("x_row", _i64), ("dt_row", _i64), ("B_row", _i64), ("C_row", _i64),
                ("z_row", _i64), ("x", _vp), ("dt", _vp), ("B", _vp), ("C", _vp), ("z", _vp), ("A", _vp), ("D", _vp),
                ("dt_bias", _vp), ("h", _vp), ("y", _vp), ("slots", _vp), ("nslots", _i32)]


class RmsnormArgs(ctypes.Structure):
    """Mirror of ``mamba3_rmsnorm_args``."""
    _fields_ = [("rows", _i64), ("dim", _i32), ("dtype", _i32), ("residual_dtype", _i32), ("qtype", _i32),
                ("qblock", _i32), ("eps", _f32), ("x_row", _i64), ("x", _vp), ("residual", _vp), ("weight", _vp),
                ("residual_out", _vp), ("y", _vp), ("q", _vp), ("qscale", _vp)]


class RmsnormBwdArgs(ctypes.Structure):
    """Mirror of ``mamba3_rmsnorm_bwd_args``."""
    _fields_ = [("rows", _i64), ("dim", _i32), ("dtype", _i32), ("residual_dtype", _i32), ("eps", _f32),
                ("dy_row", _i64), ("s", _vp), ("dy", _vp), ("dresidual_out", _vp), ("weight", _vp), ("dx", _vp),
                ("dresidual", _vp), ("dweight", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class GatedScanArgs(ctypes.Structure):
    """Mirror of ``mamba3_gated_scan_args``."""
    _fields_ = [("batch", _i32), ("seqlen", _i32), ("dim", _i32), ("dtype", _i32), ("form", _i32), ("rate", _f32),
                ("cu_seqlens", _vp), ("nseq", _i32), ("x_row", _i64), ("gate_row", _i64), ("i_row", _i64),
                ("z_row", _i64), ("x", _vp), ("gate", _vp), ("i", _vp), ("z", _vp), ("weight", _vp), ("h_in", _vp),
                ("y", _vp), ("h_out", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class GatedScanBwdArgs(ctypes.Structure):
    """Mirror of ``mamba3_gated_scan_bwd_args``."""
    _fields_ = [("fwd", GatedScanArgs), ("dy_row", _i64), ("dy", _vp), ("dh_out", _vp), ("dx", _vp), ("dgate", _vp),
                ("di", _vp), ("dz", _vp), ("dweight", _vp), ("dh_in", _vp), ("workspace", _vp),
                ("workspace_bytes", _size)]


class GatedStepArgs(ctypes.Structure):
    """Mirror of ``mamba3_gated_step_args``."""
    _fields_ = [("batch", _i32), ("dim", _i32), ("dtype", _i32), ("form", _i32), ("rate", _f32), ("x_row", _i64),
                ("gate_row", _i64), ("i_row", _i64), ("z_row", _i64), ("x", _vp), ("gate", _vp), ("i", _vp),
                ("z", _vp), ("weight", _vp), ("h", _vp), ("y", _vp), ("slots", _vp), ("nslots", _i32)]


class GroupnormArgs(ctypes.Structure):
    """Mirror of ``mamba3_groupnorm_args``."""
    _fields_ = [("rows", _i64), ("dim", _i32), ("groups", _i32), ("dtype", _i32), ("act", _i32), ("center", _i32),
                ("eps", _f32), ("x_row", _i64), ("z_row", _i64), ("x", _vp), ("z", _vp), ("weight", _vp),
                ("bias", _vp), ("y", _vp)]


class GroupnormBwdArgs(ctypes.Structure):
    """Mirror of ``mamba3_groupnorm_bwd_args``."""
    _fields_ = [("fwd", GroupnormArgs), ("dy_row", _i64), ("dy", _vp), ("dx", _vp), ("dz", _vp), ("dweight", _vp),
                ("dbias", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class StateCacheArgs(ctypes.Structure):
    """Mirror of ``mamba3_state_cache_args``."""
    _fields_ = [("n", _i32), ("values", _i32), ("dtype", _i32), ("kind", _i32), ("block", _i32), ("nslots", _i32),
                ("nentries", _i32), ("slots", _vp), ("entries", _vp), ("h", _vp), ("q", _vp), ("scale", _vp)]


# name -> (argument struct, whether there is a workspace query)
_OPS = {"conv": (ConvArgs, "fwd", False), "conv_bwd": (ConvBwdArgs, "", True), "conv_step": (ConvStepArgs, "", False),
        "selective_scan": (SelectiveScanArgs, "fwd", True), "selective_scan_bwd": (SelectiveScanBwdArgs, "", True),
        "selective_step": (SelectiveStepArgs, "", False), "rmsnorm": (RmsnormArgs, "fwd", False),
        "rmsnorm_bwd": (RmsnormBwdArgs, "", True), "gated_scan": (GatedScanArgs, "fwd", True),
        "gated_scan_bwd": (GatedScanBwdArgs, "", True), "gated_step": (GatedStepArgs, "", False),
        "groupnorm": (GroupnormArgs, "fwd", False), "groupnorm_bwd": (GroupnormBwdArgs, "", True)}
# entry points with one struct and one validation between them
_CACHE = ("state_store", "state_load")

LAYER_EXPORTS = tuple(n for op, (_, tail, ws) in _OPS.items()
                      for n in (f"mamba3_{op}_validate", f"mamba3_{op}" + (f"_{tail}" if tail else ""),
                                *([f"mamba3_{op}_workspace_size"] if ws else []))) + \
    ("mamba3_state_cache_validate", *(f"mamba3_{op}" for op in _CACHE))


def declare(l) -> None:
    """The C signatures of the layer operators on the loaded library."""
    for op, (args, tail, ws) in _OPS.items():
        f = getattr(l, f"mamba3_{op}_validate")
        f.argtypes, f.restype = [ctypes.POINTER(args)], ctypes.c_int
        f = getattr(l, f"mamba3_{op}" + (f"_{tail}" if tail else ""))
        f.argtypes, f.restype = [ctypes.POINTER(args), _vp], ctypes.c_int
        if ws:
            f = getattr(l, f"mamba3_{op}_workspace_size")
            f.argtypes, f.restype = [ctypes.POINTER(args)], _size
    for name in ("mamba3_state_cache_validate", *(f"mamba3_{op}" for op in _CACHE)):
        f = getattr(l, name)
        f.argtypes = [ctypes.POINTER(StateCacheArgs)] + ([] if name.endswith("validate") else [_vp])
        f.restype = ctypes.c_int


def _bad(what):
    raise ValueError(f"mamba3: {what}")


class _Op:
    """One entry point, called with its struct packed by its values: a single token's call takes a few
    microseconds on the GPU, and filling a ctypes structure field by field takes as long."""
    _CODES = {_i32: "i", _i64: "q", _f32: "f", _vp: "P", _size: "N"}

    def __init__(self, op):
        args, tail, ws = _OPS[op] if op in _OPS else (StateCacheArgs, "", False)
        fields = [f for _, k in args._fields_ for f in ([c for _, c in k._fields_] if hasattr(k, "_fields_") else [k])]
        inner = [k for _, k in args._fields_ if hasattr(k, "_fields_")]
        # native alignment as in C; an inner struct ends at a multiple of 8 bytes
        n = len(inner[0]._fields_) if inner else 0
        codes = [self._CODES[f] for f in fields]
        self.pack = struct.Struct("@" + "".join(codes[:n]) + ("0P" if n else "") + "".join(codes[n:]) + "0P").pack
        self.name = f"mamba3_{op}" + (f"_{tail}" if tail else "")
        l = lib()
        self.run = l[self.name]          # (a function object of its own beside the declared one)
        self.run.argtypes, self.run.restype = [ctypes.c_char_p, _vp], ctypes.c_int
        if ws:
            self.size = l[f"mamba3_{op}_workspace_size"]
            self.size.argtypes, self.size.restype = [ctypes.c_char_p], _size
        assert len(self.pack(*[0] * len(fields))) == ctypes.sizeof(args)


@functools.lru_cache(None)
def _op(op):
    return _Op(op)


def _refuse(t, shape, dtype, dev, name):
    if t.shape != shape:
        _bad(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        _bad(f"{name} must be on device {dev}, got {t.device}")
    _bad(f"{name} must be contiguous; call .contiguous()")


def _dense(t, shape, dtype, dev, name):
    """Address of a contiguous tensor of this shape and type on device number `dev`, 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, shape, dtype, dev, name)


def _rows(t, shape, lead, dtype, dev, name):
    """(device address, elements from token to token or 0) of a token array whose first `lead`
    dimensions count tokens."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, shape, dtype, dev, name)
    if t.is_contiguous():
        return t.data_ptr(), 0
    st = t.stride()
    n = 1
    for k in range(t.dim() - 1, lead - 1, -1):
        if shape[k] > 1 and st[k] != n:
            _bad(f"{name} must be dense within a token; call .contiguous()")
        n *= shape[k]
    if lead == 1:
        row = st[0] if shape[0] > 1 else n
    elif shape[1] > 1:
        row = st[1]
        if shape[0] > 1 and st[0] != row * shape[1]:
            _bad(f"{name} must have one distance between tokens; call .contiguous()")
    else:
        row = st[0] if shape[0] > 1 else n
    if row < n:
        _bad(f"{name} has overlapping tokens; call .contiguous()")
    return t.data_ptr(), row


def _new(x, dtype):
    """A new contiguous tensor of x's shape and device (empty_like costs half of empty)."""
    import torch
    if x.is_contiguous():
        return torch.empty_like(x) if x.dtype is dtype else torch.empty_like(x, dtype=dtype)
    return torch.empty(x.shape, dtype=dtype, device=x.device)


def _token(x, dims, name="x"):
    """(token dtype code, torch dtype, device number) of the leading token array."""
    if x.dim() != dims:
        _bad(f"{name} must have {dims} dimensions, got {tuple(x.shape)}")
    if not x.is_cuda:
        _bad("tensors must be in device memory")
    ty = x.dtype
    code = _dtypes().get(ty)
    if code is None:
        raise TypeError(f"token inputs must be float32 or bfloat16, got {ty}")
    return code, ty, x.get_device()


def _packed(x, cu):
    """(cu_seqlens address, nseq, sequences) of a whole-sequence call."""
    import torch
    if cu is None:
        return 0, 0, x.shape[0]
    if cu.dim() != 1 or cu.numel() < 2 or x.shape[0] != 1:
        _bad("packed batches have x [1, tokens, ...] and cu_seqlens [nseq + 1]")
    nseq = cu.numel() - 1
    return _dense(cu, cu.shape, torch.int32, x.get_device(), "cu_seqlens"), nseq, nseq


def _on(stream, x):
    """The context of a call on `stream` (a torch stream or its address): its device's and stream's
    allocations too, so that an output's memory is never one that another stream still uses."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=x.device)
    if stream.device != x.device:
        _bad(f"the stream is on {stream.device}, the tensors are on {x.device}")
    return torch.cuda.stream(stream)


def _call(op, args, dev):
    """Runs an entry point on the device's current stream."""
    import torch
    raw = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        st = op.run(args, raw)
    else:
        with torch.cuda.device(dev):
            st = op.run(args, raw)
    if st != MAMBA3_OK:
        raise Mamba3Error(st, op.name)


def _workspace(op, args, given, dev):
    """The workspace given (a contiguous uint8 tensor) or a new one, as (tensor, address, bytes); `args`
    are the call's without one."""
    import torch
    if given is None:
        need = op.size(op.pack(*args, 0, 0))
        if need == 0:
            return None, 0, 0
        given = torch.empty((need,), dtype=torch.uint8, device=dev)
        return given, given.data_ptr(), need
    return given, _dense(given, (given.numel(),), torch.uint8, dev, "workspace"), given.numel()


# ----------------------------------------------------------------------------- convolution
def _conv_args(x, weight, bias, silu, conv_in, cu_seqlens):
    import torch
    code, ty, dev = _token(x, 3)
    b, L, D = x.shape
    if weight.dim() != 2:
        _bad(f"weight must be [dim, width], got {tuple(weight.shape)}")
    W = weight.shape[1]
    cu, nseq, S = _packed(x, cu_seqlens)
    xp, xr = _rows(x, x.shape, 2, ty, dev, "x")
    a = (b, L, D, W, code, 1 if silu else 0, cu, nseq, xr, xp, _dense(weight, (D, W), torch.float32, dev, "weight"),
         _dense(bias, (D,), torch.float32, dev, "bias"), _dense(conv_in, (S, W - 1, D), ty, dev, "conv_in"))
    return a, ty, dev, S, W


def mamba3_conv_fwd(x, weight, bias=None, *, silu=True, conv_in=None, cu_seqlens=None, y=None, conv_out=None,
                    want_state=True, stream=None):
    """Short causal convolution of x [batch, seqlen, D] with weight [D, W] (fp32, W = 2..8) and bias
    [D], SiLU behind it unless silu is false. conv_in [S, W-1, D]: the inputs before each sequence's
    start (zeros if None). Returns (y, conv_out): conv_out [S, W-1, D] holds each sequence's last
    W - 1 inputs (None with want_state=False), what conv_in or mamba3_conv_step takes up."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_conv_fwd(x, weight, bias, silu=silu, conv_in=conv_in, cu_seqlens=cu_seqlens, y=y,
                                   conv_out=conv_out, want_state=want_state)
    a, ty, dev, S, W = _conv_args(x, weight, bias, silu, conv_in, cu_seqlens)
    if y is None:
        y = _new(x, ty)
    if conv_out is None and want_state:
        conv_out = torch.empty((S, max(W - 1, 0), x.shape[2]), dtype=ty, device=x.device)
    op = _op("conv")
    a = op.pack(*a, _dense(y, x.shape, ty, dev, "y"), _dense(conv_out, (S, W - 1, x.shape[2]), ty, dev, "conv_out"))
    _call(op, a, dev)
    return y, conv_out


def mamba3_conv_bwd(x, weight, bias=None, *, dy, dconv_out=None, silu=True, conv_in=None, cu_seqlens=None,
                    workspace=None, stream=None):
    """Gradients of mamba3_conv_fwd from dy and dconv_out [S, W-1, D] (None: zero): a dict of dx,
    dweight, dbias (with a bias) and dconv_in (with conv_in)."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_conv_bwd(x, weight, bias, dy=dy, dconv_out=dconv_out, silu=silu, conv_in=conv_in,
                                   cu_seqlens=cu_seqlens, workspace=workspace)
    a, ty, dev, S, W = _conv_args(x, weight, bias, silu, conv_in, cu_seqlens)
    D = x.shape[2]
    g = dict(dx=_new(x, ty), dweight=torch.empty_like(weight))
    if bias is not None:
        g["dbias"] = torch.empty_like(bias)
    if conv_in is not None:
        g["dconv_in"] = torch.empty_like(conv_in)
    yp, yr = _rows(dy, x.shape, 2, ty, dev, "dy")
    p = {k: v.data_ptr() for k, v in g.items()}
    q = (*a, 0, 0, yr, yp, _dense(dconv_out, (S, W - 1, D), ty, dev, "dconv_out"), p["dx"], p["dweight"],
         p.get("dbias", 0), p.get("dconv_in", 0))
    op = _op("conv_bwd")
    ws, wp, wn = _workspace(op, q, workspace, dev)
    _call(op, op.pack(*q, wp, wn), dev)
    return g


def _slots(slots, batch, state, dev):
    """(address, pool size, states) of a step's slot table."""
    import torch
    if slots is None:
        return 0, 0, batch
    return _dense(slots, (batch,), torch.int32, dev, "slots"), state.shape[0], state.shape[0]


def mamba3_conv_step(x, weight, bias=None, *, conv, silu=True, slots=None, y=None, stream=None):
    """One token x [batch, D] through the convolution; conv [batch, W-1, D] moves on by one input in
    place. With slots (int32 [batch] on the device) conv is a pool [nslots, W-1, D]; rows with a slot
    outside the pool are skipped (their y rows stay as they were). Returns y."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_conv_step(x, weight, bias, conv=conv, silu=silu, slots=slots, y=y)
    code, ty, dev = _token(x, 2)
    b, D = x.shape
    if weight.dim() != 2:
        _bad(f"weight must be [dim, width], got {tuple(weight.shape)}")
    W = weight.shape[1]
    if y is None:
        y = _new(x, ty)
    sp, ns, states = _slots(slots, b, conv, dev)
    xp, xr = _rows(x, x.shape, 1, ty, dev, "x")
    op = _op("conv_step")
    a = op.pack(b, D, W, code, 1 if silu else 0, xr, xp, _dense(weight, (D, W), torch.float32, dev, "weight"),
                _dense(bias, (D,), torch.float32, dev, "bias"), _dense(conv, (states, W - 1, D), ty, dev, "conv"),
                _dense(y, (b, D), ty, dev, "y"), sp, ns)
    _call(op, a, dev)
    return y


# ----------------------------------------------------------------------------- selective scan
def _sel_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, h_in, cu_seqlens):
    import torch
    code, ty, dev = _token(x, 3)
    b, L, dim = x.shape
    if B.dim() != 4 or A.dim() != 2:
        _bad(f"A must be [dim, dstate] and B [batch, seqlen, groups, dstate], got {tuple(A.shape)}, {tuple(B.shape)}")
    G, N = B.shape[2], B.shape[3]
    cu, nseq, S = _packed(x, cu_seqlens)
    xp, xr = _rows(x, x.shape, 2, ty, dev, "x")
    dp, dr = _rows(dt, x.shape, 2, ty, dev, "dt")
    zp, zr = _rows(z, x.shape, 2, ty, dev, "z")
    bp, br = _rows(B, (b, L, G, N), 2, ty, dev, "B")
    cp, cr = _rows(C, (b, L, G, N), 2, ty, dev, "C")
    f = torch.float32
    a = (b, L, dim, N, G, code, 1 if dt_softplus else 0, cu, nseq, xr, dr, br, cr, zr, xp, dp, bp, cp, zp,
         _dense(A, (dim, N), f, dev, "A"), _dense(D, (dim,), f, dev, "D"), _dense(dt_bias, (dim,), f, dev, "dt_bias"),
         _dense(h_in, (S, dim, N), f, dev, "h_in"))
    return a, ty, dev, S, N


def mamba3_selective_scan_fwd(x, dt, A, B, C, D=None, *, z=None, dt_bias=None, dt_softplus=False, h_in=None,
                              cu_seqlens=None, y=None, h_out=None, want_state=True, workspace=None, stream=None):
    """Selective scan: h_t = exp(s_t A) h_{t-1} + s_t x_t B_t, y_t = (C_t h_t + D x_t) SiLU(z_t), with
    s_t = dt_t + dt_bias (softplus of it with dt_softplus). x, dt, z [batch, seqlen, dim]; B, C
    [batch, seqlen, G, N] (N <= 128); A [dim, N], D, dt_bias [dim], h_in [S, dim, N] fp32. Returns (y,
    h_out [S, dim, N] or None with want_state=False)."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_selective_scan_fwd(x, dt, A, B, C, D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus,
                                             h_in=h_in, cu_seqlens=cu_seqlens, y=y, h_out=h_out, want_state=want_state,
                                             workspace=workspace)
    a, ty, dev, S, N = _sel_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, h_in, cu_seqlens)
    if y is None:
        y = _new(x, ty)
    if h_out is None and want_state:
        h_out = torch.empty((S, x.shape[2], N), dtype=torch.float32, device=x.device)
    a += (_dense(y, x.shape, ty, dev, "y"), _dense(h_out, (S, x.shape[2], N), torch.float32, dev, "h_out"))
    op = _op("selective_scan")
    ws, wp, wn = _workspace(op, a, workspace, dev)
    _call(op, op.pack(*a, wp, wn), dev)
    return y, h_out


def mamba3_selective_scan_bwd(x, dt, A, B, C, D=None, *, dy, dh_out=None, z=None, dt_bias=None, dt_softplus=False,
                              h_in=None, cu_seqlens=None, want_dh_in=None, workspace=None, stream=None):
    """Gradients of mamba3_selective_scan_fwd from dy and dh_out [S, dim, N] (None: zero): a dict of dx,
    ddt, dB, dC, dA, and dD, dz, ddt_bias, dh_in where the input exists (dh_in always with
    want_dh_in=True)."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_selective_scan_bwd(x, dt, A, B, C, D, dy=dy, dh_out=dh_out, z=z, dt_bias=dt_bias,
                                             dt_softplus=dt_softplus, h_in=h_in, cu_seqlens=cu_seqlens,
                                             want_dh_in=want_dh_in, workspace=workspace)
    a, ty, dev, S, N = _sel_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, h_in, cu_seqlens)
    dim = x.shape[2]
    g = dict(dx=_new(x, ty), ddt=_new(x, ty),
             dB=_new(B, ty), dC=_new(B, ty),
             dA=torch.empty_like(A))
    if D is not None:
        g["dD"] = torch.empty_like(D)
    if z is not None:
        g["dz"] = _new(x, ty)
    if dt_bias is not None:
        g["ddt_bias"] = torch.empty_like(dt_bias)
    if h_in is not None if want_dh_in is None else want_dh_in:
        g["dh_in"] = torch.empty((S, dim, N), dtype=torch.float32, device=x.device)
    yp, yr = _rows(dy, x.shape, 2, ty, dev, "dy")
    p = {k: v.data_ptr() for k, v in g.items()}
    q = (*a, 0, 0, 0, 0, yr, yp, _dense(dh_out, (S, dim, N), torch.float32, dev, "dh_out"),
         *[p.get(k, 0) for k in ("dx", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias", "dh_in")])
    op = _op("selective_scan_bwd")
    ws, wp, wn = _workspace(op, q, workspace, dev)
    _call(op, op.pack(*q, wp, wn), dev)
    return g


def mamba3_selective_step(x, dt, A, B, C, D=None, *, h, z=None, dt_bias=None, dt_softplus=False, slots=None, y=None,
                          stream=None):
    """One token of the selective scan: x, dt, z [batch, dim], B, C [batch, G, N]; h [batch, dim, N]
    (fp32) is updated in place. With slots (int32 [batch] on the device) h is a pool [nslots, dim,
    N]; rows with a slot outside the pool are skipped (their y rows stay as they were). Returns y."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_selective_step(x, dt, A, B, C, D, h=h, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus,
                                         slots=slots, y=y)
    code, ty, dev = _token(x, 2)
    b, dim = x.shape
    if B.dim() != 3 or A.dim() != 2:
        _bad(f"A must be [dim, dstate] and B [batch, groups, dstate], got {tuple(A.shape)}, {tuple(B.shape)}")
    G, N = B.shape[1], B.shape[2]
    if y is None:
        y = _new(x, ty)
    f = torch.float32
    sp, ns, states = _slots(slots, b, h, dev)
    xp, xr = _rows(x, x.shape, 1, ty, dev, "x")
    dp, dr = _rows(dt, x.shape, 1, ty, dev, "dt")
    zp, zr = _rows(z, x.shape, 1, ty, dev, "z")
    bp, br = _rows(B, (b, G, N), 1, ty, dev, "B")
    cp, cr = _rows(C, (b, G, N), 1, ty, dev, "C")
    op = _op("selective_step")
    a = op.pack(b, dim, N, G, code, 1 if dt_softplus else 0, xr, dr, br, cr, zr, xp, dp, bp, cp, zp,
                _dense(A, (dim, N), f, dev, "A"), _dense(D, (dim,), f, dev, "D"),
                _dense(dt_bias, (dim,), f, dev, "dt_bias"), _dense(h, (states, dim, N), f, dev, "h"),
                _dense(y, (b, dim), ty, dev, "y"), sp, ns)
    _call(op, a, dev)
    return y


# ----------------------------------------------------------------------------- RMS norm
def mamba3_rmsnorm_fwd(x, weight=None, *, residual=None, eps=1e-5, y=None, residual_out=None, want_y=True, quant=None,
                       qblock=128, stream=None):
    """s = x + residual and its RMS norm times weight, over the last dimension of x [..., dim] (bf16 or
    fp32; residual in x's type or fp32). Returns a dict of y (unless want_y is false), residual (s, in
    residual's type; residual_out, which may be residual itself, if given) where there is a residual,
    and with quant "e4m3" or "int8" q [..., dim] and scale [..., blocks] (fp32, the norm is q * scale
    up to rounding): one scale for each qblock (32, 64, 128, 256) channels, or a row with qblock 0."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_rmsnorm_fwd(x, weight, residual=residual, eps=eps, y=y, residual_out=residual_out,
                                      want_y=want_y, quant=quant, qblock=qblock)
    dim = x.shape[-1] if x.dim() else 0
    flat = x if x.dim() == 2 else x.reshape(-1, dim) if dim else x
    code, ty, dev = _token(flat, 2)
    rows = flat.shape[0]
    rt = residual.dtype if residual is not None else residual_out.dtype if residual_out is not None else ty
    if rt not in _dtypes():
        raise TypeError(f"residual must be float32 or bfloat16, got {rt}")
    if not want_y and quant is None:
        _bad("nothing to compute: want_y is false and quant is None")
    out = {}
    if residual is not None and residual_out is None:
        residual_out = _new(x, rt)
    if residual_out is not None:
        out["residual"] = residual_out
    if want_y or y is not None:
        if y is None:
            y = _new(x, ty)
        out["y"] = y
    qp = sp = 0
    qcode = 0
    if quant is not None:
        if quant not in _qtypes():
            _bad(f"quant must be one of {sorted(_qtypes())}, got {quant!r}")
        qcode, qt = _qtypes()[quant]
        blocks = 1 if qblock <= 0 or qblock >= dim else -(-dim // qblock)
        out["q"] = _new(x, qt)
        out["scale"] = torch.empty((*x.shape[:-1], blocks), dtype=torch.float32, device=x.device)
        qp, sp = out["q"].data_ptr(), out["scale"].data_ptr()
    xp, xr = _rows(flat, (rows, dim), 1, ty, dev, "x")
    op = _op("rmsnorm")
    a = op.pack(rows, dim, code, _dtypes()[rt], qcode, qblock, eps, xr, xp,
                _dense(residual, x.shape, rt, dev, "residual"), _dense(weight, (dim,), torch.float32, dev, "weight"),
                _dense(residual_out, x.shape, rt, dev, "residual_out"), _dense(y, x.shape, ty, dev, "y"), qp, sp)
    _call(op, a, dev)
    return out


def mamba3_rmsnorm_bwd(s, weight=None, *, dy, dresidual_out=None, eps=1e-5, want_dx=True, workspace=None, stream=None):
    """Gradients of mamba3_rmsnorm_fwd from s (its residual output, or x without a residual), dy (of y)
    and dresidual_out (of the residual output, s's type; None: zero): a dict of dresidual (s's type),
    dx (dy's type: the same tensor where the types are equal) and dweight (with a weight)."""
    import torch
    if stream is not None:
        with _on(stream, s):
            return mamba3_rmsnorm_bwd(s, weight, dy=dy, dresidual_out=dresidual_out, eps=eps, want_dx=want_dx,
                                      workspace=workspace)
    dim = s.shape[-1] if s.dim() else 0
    if dy.shape != s.shape:
        _bad(f"dy must have shape {tuple(s.shape)}, got {tuple(dy.shape)}")
    flat = dy if dy.dim() == 2 else dy.reshape(-1, dim) if dim else dy
    code, ty, dev = _token(flat, 2, "dy")
    rows, rt = flat.shape[0], s.dtype
    if rt not in _dtypes():
        raise TypeError(f"s must be float32 or bfloat16, got {rt}")
    g = dict(dresidual=_new(s, rt))
    dx = None
    if want_dx:
        if rt == ty:
            g["dx"] = g["dresidual"]
        else:
            dx = g["dx"] = _new(s, ty)
    if weight is not None:
        g["dweight"] = torch.empty_like(weight)
    yp, yr = _rows(flat, (rows, dim), 1, ty, dev, "dy")
    op = _op("rmsnorm_bwd")
    a = (rows, dim, code, _dtypes()[rt], eps, yr, _dense(s, s.shape, rt, dev, "s"), yp,
         _dense(dresidual_out, s.shape, rt, dev, "dresidual_out"), _dense(weight, (dim,), torch.float32, dev, "weight"),
         dx.data_ptr() if dx is not None else 0, g["dresidual"].data_ptr(),
         g["dweight"].data_ptr() if weight is not None else 0)
    ws, wp, wn = _workspace(op, a, workspace, dev)
    _call(op, op.pack(*a, wp, wn), dev)
    return g


# ----------------------------------------------------------------------------- gated linear recurrence
def _form(form, rate):
    if form not in _FORMS:
        _bad(f"form must be one of {sorted(_FORMS)}, got {form!r}")
    return _FORMS[form], float(rate)


def _gated_args(x, gate, weight, form, rate, i, z, h_in, cu_seqlens):
    import torch
    code, ty, dev = _token(x, 3)
    b, L, D = x.shape
    fc, rate = _form(form, rate)
    cu, nseq, S = _packed(x, cu_seqlens)
    xp, xr = _rows(x, x.shape, 2, ty, dev, "x")
    gp, gr = _rows(gate, x.shape, 2, ty, dev, "gate")
    ip, ir = _rows(i, x.shape, 2, ty, dev, "i")
    zp, zr = _rows(z, x.shape, 2, ty, dev, "z")
    f = torch.float32
    a = (b, L, D, code, fc, rate, cu, nseq, xr, gr, ir, zr, xp, gp, ip, zp, _dense(weight, (D,), f, dev, "weight"),
         _dense(h_in, (S, D), f, dev, "h_in"))
    return a, ty, dev, S


def mamba3_gated_scan_fwd(x, gate, weight=None, *, form="decay", rate=8.0, i=None, z=None, h_in=None, cu_seqlens=None,
                          y=None, h_out=None, want_state=True, workspace=None, stream=None):
    """Gated linear recurrence: h_t = a_t h_{t-1} + u_t sigmoid(i_t) x_t (x_t alone without i), y_t = h_t
    (h_t SiLU(z_t) with z). form "decay": a = exp(-rate softplus(weight) sigmoid(gate)), u = sqrt(1 -
    a^2); "forget": a = l + (1 - l) sigmoid(gate) with the least decay l = weight (0 without), u = 1 - a.
    x, gate, i, z [batch, seqlen, D]; weight [D], h_in [S, D] fp32. Returns (y, h_out [S, D] or None with
    want_state=False)."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_gated_scan_fwd(x, gate, weight, form=form, rate=rate, i=i, z=z, h_in=h_in,
                                         cu_seqlens=cu_seqlens, y=y, h_out=h_out, want_state=want_state,
                                         workspace=workspace)
    a, ty, dev, S = _gated_args(x, gate, weight, form, rate, i, z, h_in, cu_seqlens)
    if y is None:
        y = _new(x, ty)
    if h_out is None and want_state:
        h_out = torch.empty((S, x.shape[2]), dtype=torch.float32, device=x.device)
    a += (_dense(y, x.shape, ty, dev, "y"), _dense(h_out, (S, x.shape[2]), torch.float32, dev, "h_out"))
    op = _op("gated_scan")
    ws, wp, wn = _workspace(op, a, workspace, dev)
    _call(op, op.pack(*a, wp, wn), dev)
    return y, h_out


def mamba3_gated_scan_bwd(x, gate, weight=None, *, dy, dh_out=None, form="decay", rate=8.0, i=None, z=None, h_in=None,
                          cu_seqlens=None, want_dh_in=None, workspace=None, stream=None):
    """Gradients of mamba3_gated_scan_fwd from dy and dh_out [S, D] (None: zero): a dict of dx, dgate, and di,
    dz, dweight, dh_in where the input exists (dh_in always with want_dh_in=True)."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_gated_scan_bwd(x, gate, weight, dy=dy, dh_out=dh_out, form=form, rate=rate, i=i, z=z,
                                         h_in=h_in, cu_seqlens=cu_seqlens, want_dh_in=want_dh_in, workspace=workspace)
    a, ty, dev, S = _gated_args(x, gate, weight, form, rate, i, z, h_in, cu_seqlens)
    g = dict(dx=_new(x, ty), dgate=_new(x, ty))
    if i is not None:
        g["di"] = _new(x, ty)
    if z is not None:
        g["dz"] = _new(x, ty)
    if weight is not None:
        g["dweight"] = torch.empty_like(weight)
    if h_in is not None if want_dh_in is None else want_dh_in:
        g["dh_in"] = torch.empty((S, x.shape[2]), dtype=torch.float32, device=x.device)
    yp, yr = _rows(dy, x.shape, 2, ty, dev, "dy")
    p = {k: v.data_ptr() for k, v in g.items()}
    q = (*a, 0, 0, 0, 0, yr, yp, _dense(dh_out, (S, x.shape[2]), torch.float32, dev, "dh_out"),
         *[p.get(k, 0) for k in ("dx", "dgate", "di", "dz", "dweight", "dh_in")])
    op = _op("gated_scan_bwd")
    ws, wp, wn = _workspace(op, q, workspace, dev)
    _call(op, op.pack(*q, wp, wn), dev)
    return g


def mamba3_gated_step(x, gate, weight=None, *, h, form="decay", rate=8.0, i=None, z=None, slots=None, y=None,
                      stream=None):
    """One token of the gated linear recurrence: x, gate, i, z [batch, D]; h [batch, D] (fp32) is updated
    in place. With slots (int32 [batch] on the device) h is a pool [nslots, D]; rows with a slot outside the
    pool are skipped (their y rows stay as they were). Returns y."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_gated_step(x, gate, weight, h=h, form=form, rate=rate, i=i, z=z, slots=slots, y=y)
    code, ty, dev = _token(x, 2)
    b, D = x.shape
    fc, rate = _form(form, rate)
    if y is None:
        y = _new(x, ty)
    f = torch.float32
    sp, ns, states = _slots(slots, b, h, dev)
    xp, xr = _rows(x, x.shape, 1, ty, dev, "x")
    gp, gr = _rows(gate, x.shape, 1, ty, dev, "gate")
    ip, ir = _rows(i, x.shape, 1, ty, dev, "i")
    zp, zr = _rows(z, x.shape, 1, ty, dev, "z")
    op = _op("gated_step")
    a = op.pack(b, D, code, fc, rate, xr, gr, ir, zr, xp, gp, ip, zp, _dense(weight, (D,), f, dev, "weight"),
                _dense(h, (states, D), f, dev, "h"), _dense(y, (b, D), ty, dev, "y"), sp, ns)
    _call(op, a, dev)
    return y


# ----------------------------------------------------------------------------- group norm
def _groupnorm_args(x, weight, bias, groups, z, act, center, eps):
    import torch
    dim = x.shape[-1] if x.dim() else 0
    if act not in _ACTS:
        _bad(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    flat = x if x.dim() == 2 else x.reshape(-1, dim) if dim else x
    code, ty, dev = _token(flat, 2)
    rows = flat.shape[0]
    if z is not None and z.shape != x.shape:
        _bad(f"z must have shape {tuple(x.shape)}, got {tuple(z.shape)}")
    xp, xr = _rows(flat, (rows, dim), 1, ty, dev, "x")
    # (kept until the call: a view of more dimensions may have been copied)
    zf = z if z is None or z.dim() == 2 else z.reshape(-1, dim)
    zp, zr = _rows(zf, (rows, dim), 1, ty, dev, "z")
    f = torch.float32
    a = (rows, dim, groups, code, _ACTS[act], 1 if center else 0, eps, xr, zr, xp, zp,
         _dense(weight, (dim,), f, dev, "weight"), _dense(bias, (dim,), f, dev, "bias"))
    return a, ty, dev, (flat, zf)


def mamba3_groupnorm_fwd(x, weight=None, bias=None, *, groups, z=None, act="none", center=True, eps=1e-5, y=None,
                         stream=None):
    """Group norm over the last dimension of x [..., dim], whose channels are `groups` groups of consecutive
    ones with statistics of their own row: v = (t - mean) / sqrt(var + eps) weight + bias (center=False: t /
    sqrt(mean t^2 + eps) weight + bias), t = x. act "none": v; "silu": v sigmoid(v); "gate": v SiLU(z);
    "pregate": v of t = x SiLU(z). weight, bias [dim] fp32. Returns y."""
    if stream is not None:
        with _on(stream, x):
            return mamba3_groupnorm_fwd(x, weight, bias, groups=groups, z=z, act=act, center=center, eps=eps, y=y)
    a, ty, dev, kept = _groupnorm_args(x, weight, bias, groups, z, act, center, eps)
    if y is None:
        y = _new(x, ty)
    op = _op("groupnorm")
    _call(op, op.pack(*a, _dense(y, x.shape, ty, dev, "y")), dev)
    return y


def mamba3_groupnorm_bwd(x, weight=None, bias=None, *, dy, groups, z=None, act="none", center=True, eps=1e-5,
                         workspace=None, stream=None):
    """Gradients of mamba3_groupnorm_fwd from dy: a dict of dx, and dz, dweight, dbias where the input
    exists."""
    import torch
    if stream is not None:
        with _on(stream, x):
            return mamba3_groupnorm_bwd(x, weight, bias, dy=dy, groups=groups, z=z, act=act, center=center, eps=eps,
                                        workspace=workspace)
    if dy.shape != x.shape:
        _bad(f"dy must have shape {tuple(x.shape)}, got {tuple(dy.shape)}")
    a, ty, dev, kept = _groupnorm_args(x, weight, bias, groups, z, act, center, eps)
    g = dict(dx=_new(x, ty))
    if z is not None:
        g["dz"] = _new(x, ty)
    if weight is not None:
        g["dweight"] = torch.empty_like(weight)
    if bias is not None:
        g["dbias"] = torch.empty_like(bias)
    df = dy if dy.dim() == 2 else dy.reshape(-1, x.shape[-1])
    yp, yr = _rows(df, kept[0].shape, 1, ty, dev, "dy")
    p = {k: v.data_ptr() for k, v in g.items()}
    q = (*a, 0, yr, yp, *[p.get(k, 0) for k in ("dx", "dz", "dweight", "dbias")])
    op = _op("groupnorm_bwd")
    ws, wp, wn = _workspace(op, q, workspace, dev)
    _call(op, op.pack(*q, wp, wn), dev)
    return g


# ----------------------------------------------------------------------------- state cache
def _cache_index(t, name, dev):
    import torch
    if t is None:
        return 0, None
    if t.dim() != 1:
        _bad(f"{name} must have one dimension, got {tuple(t.shape)}")
    return _dense(t, t.shape, torch.int32, dev, name), t.shape[0]


def _cache_call(op, h, kind, block, slots, entries, q, scale):
    import torch
    if kind not in _kinds():
        _bad(f"kind must be one of {sorted(_kinds())}, got {kind!r}")
    if h.dim() < 2:
        _bad(f"h must be [slots, ...], got {tuple(h.shape)}")
    if not h.is_cuda:
        _bad("tensors must be in device memory")
    ty = h.dtype
    code = _dtypes().get(ty)
    if code is None:
        raise TypeError(f"states must be float32 or bfloat16, got {ty}")
    dev = h.get_device()
    kc, qt = _kinds()[kind]
    values = math.prod(h.shape[1:])
    if values < 1:
        _bad(f"a state has no values: {tuple(h.shape)}")
    if block not in (32, 64, 128, 256):
        _bad(f"block must be 32, 64, 128 or 256, got {block}")
    sp, n = _cache_index(slots, "slots", dev)
    ep, m = _cache_index(entries, "entries", dev)
    if n is not None and m is not None and n != m:
        _bad(f"slots and entries must be equally many, got {n} and {m}")
    bytes_, blocks = (values + 1) // 2 if kind == "int4" else values, -(-values // block)
    if n is None:
        n = m if m is not None else h.shape[0]
    if q is None:
        if m is not None:
            _bad("entries are places in a cache: q and scale are needed with them")
        q = torch.empty((n, bytes_), dtype=qt, device=h.device)
        scale = torch.empty((n, blocks), dtype=torch.float32, device=h.device)
    if q.dim() != 2:
        _bad(f"q must be [entries, bytes of a state], got {tuple(q.shape)}")
    nentries = q.shape[0]
    if (slots is None and h.shape[0] < n) or (entries is None and nentries < n):
        _bad(f"{n} rows do not lie in {h.shape[0]} slots and {nentries} entries")
    o = _op(op)
    a = o.pack(n, values, code, kc, block, h.shape[0], nentries, sp, ep, _dense(h, h.shape, ty, dev, "h"),
               _dense(q, (nentries, bytes_), qt, dev, "q"),
               _dense(scale, (nentries, blocks), torch.float32, dev, "scale"))
    _call(o, a, dev)
    return q, scale


def mamba3_state_store(h, *, kind="int8", block=64, slots=None, entries=None, q=None, scale=None, stream=None):
    """Writes states of the pool h [nslots, ...] (fp32 or bf16) into a cache in 8 or 4 bits: state slots[k] (k
    without slots) into entry entries[k] (k without entries) of q and scale, with one scale for each `block`
    (32, 64, 128, 256) consecutive values. kind "e4m3" and "int8": q [nentries, values]; "int4": uint8
    [nentries, (values + 1) // 2], two values a byte; scale [nentries, blocks] fp32. Without q a
    cache of as many entries as rows is made. slots, entries: int32 [n] on the device; rows with either
    outside its range are skipped, and rows name different entries. Returns (q, scale)."""
    if stream is not None:
        with _on(stream, h):
            return mamba3_state_store(h, kind=kind, block=block, slots=slots, entries=entries, q=q, scale=scale)
    if (q is None) != (scale is None):
        _bad("q and scale come together")
    return _cache_call("state_store", h, kind, block, slots, entries, q, scale)


def mamba3_state_load(q, scale, *, h, kind="int8", block=64, slots=None, entries=None, stream=None):
    """Reads cache entries back into the pool h [nslots, ...]: entry entries[k] into state slots[k], as
    mamba3_state_store wrote them; rows name different slots. Other states stay as they were. Returns h."""
    if stream is not None:
        with _on(stream, h):
            return mamba3_state_load(q, scale, h=h, kind=kind, block=block, slots=slots, entries=entries)
    if q is None or scale is None:
        _bad("q and scale are needed")
    if slots is None and entries is None:
        # (whole caches: as many as there are of both)
        if q.dim() == 2 and h.dim() and q.shape[0] != h.shape[0]:
            _bad(f"{q.shape[0]} entries and {h.shape[0]} slots: slots or entries are needed")
    _cache_call("state_load", h, kind, block, slots, entries, q, scale)
    return h
