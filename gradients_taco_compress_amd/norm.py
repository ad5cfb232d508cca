"""Binding of libtaco_norm (include/taco_norm.h) and libtaco_rms
(include/taco_rms.h): layer norm for training, with an 8-bit checkpoint of the
normalised activation that serves both the norm's backward pass and the weight
gradient of the linear layer behind it; and root-mean-square norm with the
residual's addition, for training and into 8 bits.

Three layers:

* ``taco_norm_*`` and ``taco_rms_*``: the C ABIs with the same names and
  arguments (device pointers and stream handles as ints).
* ``layer_norm``, ``layer_norm_backward``, ``layer_norm_checkpoint``,
  ``layer_norm_checkpoint_backward``, ``checkpoint_weight_grad``, ``rms_norm``,
  ``rms_norm_mx``, ``rms_norm_backward``: the same calls on torch tensors,
  allocating outputs (and workspaces) when none are given and launching on
  torch's current stream.
* ``norm``, ``rms`` and ``norm_linear``: autograd functions made of them.
  ``norm_linear`` is a layer norm and the linear layer behind it; it keeps one
  byte per activation element for its backward pass instead of the norm's
  input and output (four bytes in bf16).

Activations are bf16, fp16 or float32 tensors [..., hidden] whose rows are
contiguous and evenly spaced (a column slice of a wider tensor is fine).
Norm parameters are of the activations' type or float32.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import TacoError, taco_status_string  # noqa: F401  (torch's HIP runtime is loaded first)

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtaco_norm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libtaco_norm.so is not built ({LIB_PATH} missing); run "
        "`python gradients_taco_compress_amd/build.py` (there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

# The usual calls, without the interpreter between them and the C ABI: each
# function takes tensors only and returns None for what is not usual (the code
# below then takes over, and words the errors).
try:
    from . import _norm_torch as _fast
except ImportError as e:
    raise ImportError(f"the torch module of libtaco_norm is not built ({e}); run "
                      "`python gradients_taco_compress_amd/build.py`") from e

_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_STATUS = ctypes.c_int
_SIGNATURES = {
    "taco_norm_checkpoint_scale": ([_I64], _F32),
    "taco_norm_forward": ([_P, _I64, _I64, _I64, _I32, _P, _P, _I32, _F32, _P, _I64, _P, _P, _P],
                          _STATUS),
    "taco_norm_checkpoint": ([_P, _I64, _I64, _I64, _I32, _P, _P, _I32, _F32, _P, _I64, _P, _P,
                              _P], _STATUS),
    "taco_norm_backward_workspace": ([_I64, _I64], _I64),
    "taco_norm_backward": ([_P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I32, _I32, _P, _I64, _P,
                            _P, _P, _I64, _P], _STATUS),
    "taco_norm_checkpoint_backward": ([_P, _I64, _P, _P, _P, _I64, _I64, _I32, _I32, _P, _I64, _P,
                                       _P, _P, _I64, _P], _STATUS),
    "taco_norm_weight_grad_workspace": ([_P, _I64, _P, _I64, _I64, _I64], _I64),
    "taco_norm_weight_grad": ([_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _P, _I32, _P, _I32, _I32,
                               _P, _P, _I64, _P], _STATUS),
}
#: Symbols the library exports (checked against include/taco_norm.h).
EXPORTS = tuple(_SIGNATURES)
for _name, (_args, _res) in _SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes, _fn.restype = _args, _res
    globals()[_name] = _fn

# Root-mean-square norm is a library of its own (include/taco_rms.h): where it is not
# built, layer norm works all the same.
RMS_LIB_PATH = os.path.join(PKG, "libtaco_rms.so")


class _NotBuilt:
    """In the place of a library that is missing: any use of it says so."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        def call(*args):
            raise ImportError(f"{self._why}; run `python gradients_taco_compress_amd/build.py` "
                              "(there is no CPU fallback)")
        return call


def _load_rms():
    """(the library, its torch module)."""
    if not os.path.exists(RMS_LIB_PATH):
        missing = _NotBuilt(f"libtaco_rms.so is not built ({RMS_LIB_PATH} missing)")
        return missing, missing
    lib = ctypes.CDLL(RMS_LIB_PATH)
    try:
        from . import _rms_torch
    except ImportError as e:
        missing = _NotBuilt(f"the torch module of libtaco_rms is not built ({e})")
        return missing, missing
    return lib, _rms_torch


_rms, _fast_rms = _load_rms()
_RMS_SIGNATURES = {
    "taco_rms_forward": ([_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _I32, _F32, _P, _I64, _P,
                          _I64, _P, _P], _STATUS),
    "taco_rms_mx": ([_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _I32, _F32, _P, _P, _P, _I64, _P],
                    _STATUS),
    "taco_rms_backward_workspace": ([_I64, _I64], _I64),
    "taco_rms_backward": ([_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _I32, _I32, _P,
                           _I64, _P, _P, _I64, _P], _STATUS),
}
#: Symbols that library exports (checked against include/taco_rms.h).
RMS_EXPORTS = tuple(_RMS_SIGNATURES)
for _name, (_args, _res) in _RMS_SIGNATURES.items():
    _fn = getattr(_rms, _name)
    _fn.argtypes, _fn.restype = _args, _res
    globals()[_name] = _fn

#: taco_norm_dtype of the torch types.
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
#: Widest row.
MAX_HIDDEN = 1048576


def checkpoint_scale(hidden: int) -> float:
    """S of a checkpoint with rows of ``hidden`` elements: the normalised
    activation is ``taco.decode(codes) / S``."""
    s = _lib.taco_norm_checkpoint_scale(hidden)
    if s == 0.0:
        raise TacoError(2, "taco_norm_checkpoint_scale")
    return s


# ------------------------------------------------------------- arguments --

def _check(status: int, what: str) -> None:
    if status != 0:
        raise TacoError(status, what)


def _device_tensor(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA/HIP torch tensor")


def _pitch(t, name, dtype=None):
    """(rows, row length, elements between rows) of a tensor [..., hidden]."""
    _device_tensor(t, name)
    if dtype is None:
        if t.dtype not in DTYPES:
            raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() == 0:
        raise ValueError(f"{name}: expected a tensor with at least one dimension")
    hidden = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // hidden if hidden else 0), hidden, hidden
    if t.numel() == 0:
        return 0, hidden, hidden
    if hidden > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: rows must be contiguous (last stride 1)")
    rows, pitch = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if pitch is None:
            pitch = stride
        elif stride != pitch * rows:
            raise ValueError(f"{name}: rows must be evenly spaced")
        rows *= size
    pitch = hidden if pitch is None else pitch
    if pitch < hidden:
        raise ValueError(f"{name}: rows overlap (an expanded tensor?)")
    return rows, hidden, pitch


def _param(t, hidden, dtype, name):
    """Checks a norm parameter; returns its device pointer (0 for None)."""
    if t is None:
        return 0
    _device_tensor(t, name)
    if t.dtype != dtype and t.dtype != torch.float32:
        raise TypeError(f"{name} must be {dtype} or torch.float32, got {t.dtype}")
    if t.numel() != hidden or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {hidden} elements")
    return t.data_ptr()


def _param_type(weight, bias, dtype):
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight and bias must have one type, got {weight.dtype} and {bias.dtype}")
    p = weight if weight is not None else bias
    return dtype if p is None else p.dtype


def _vector(t, n, name, dtype=torch.float32):
    _device_tensor(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    return t.data_ptr()


def _codes(t, rows, hidden):
    """Checks a checkpoint [..., hidden] of `rows` rows; returns its device
    pointer.  (Not by its size alone: a [hidden, rows] tensor has that, too.)"""
    p = _vector(t, rows * hidden, "codes", torch.uint8)
    if t.dim() == 0 or t.shape[-1] != hidden:
        raise ValueError(f"codes must hold rows of {hidden}, got {list(t.shape)}")
    return p


class _Launch:
    """Where a call runs: its stream, and the allocation of what it returns.

    With a stream other than torch's current one, outputs and workspaces come
    from that stream's memory (memory of the current stream may still be in
    use by earlier work there), and every tensor of the call is recorded on the
    stream it was not allocated on."""

    def __init__(self, stream, tensors):
        first = tensors[0].device
        for t in tensors:
            if t is not None and t.device != first:
                devs = sorted({str(u.device) for u in tensors if u is not None})
                raise ValueError(f"tensors are on different devices: {devs}")
        current = torch.cuda.current_stream(first)
        if stream is not None and stream.device != first:
            raise ValueError(f"stream is on {stream.device}, tensors on {first}")
        self.device = first
        self.current = current
        self.stream = current if stream is None else stream
        self.other = self.stream != current
        if self.other:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)

    def empty(self, shape, dtype):
        if not self.other:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(self.current)
        return t

    def workspace(self, nbytes):
        if nbytes <= 0:
            return None
        with torch.cuda.stream(self.stream) if self.other else contextlib.nullcontext():
            return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def call(self, fn, what, *args):
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                _check(fn(*args, self.stream.cuda_stream), what)
        else:
            _check(fn(*args, self.stream.cuda_stream), what)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# -------------------------------------------------------------- operators --

def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, mean=None, rstd=None,
               stream=None):
    """Layer norm over the last dimension: (y, mean, rstd), the statistics
    float32 [rows], as the backward pass takes them."""
    if out is None and mean is None and rstd is None and stream is None:
        done = _fast.layer_norm(x, weight, bias, eps)
        if done is not None:
            return done
    rows, hidden, ldx = _pitch(x, "x")
    w, b = _param(weight, hidden, x.dtype, "weight"), _param(bias, hidden, x.dtype, "bias")
    ptype = _param_type(weight, bias, x.dtype)
    at = _Launch(stream, (x, weight, bias, out, mean, rstd))
    out = at.empty(x.shape, x.dtype) if out is None else out
    mean = at.empty(rows, torch.float32) if mean is None else mean
    rstd = at.empty(rows, torch.float32) if rstd is None else rstd
    ldy = _same_rows(out, "out", x.dtype, rows, hidden)
    at.call(_lib.taco_norm_forward, "taco_norm_forward", x.data_ptr(), ldx, rows, hidden,
            DTYPES[x.dtype], w, b, DTYPES[ptype], eps, out.data_ptr(), ldy,
            _vector(mean, rows, "mean"), _vector(rstd, rows, "rstd"))
    return out, mean, rstd


def _same_rows(t, name, dtype, rows, hidden):
    r, h, ld = _pitch(t, name, dtype)
    if (r, h) != (rows, hidden):
        raise ValueError(f"{name} must hold {rows} rows of {hidden}, got {r} of {h}")
    return ld


def layer_norm_checkpoint(x, weight=None, bias=None, eps: float = 1e-5, out=None, codes=None,
                          rstd=None, stream=None):
    """Layer norm that also writes its 8-bit checkpoint: (y, codes, rstd) with
    codes uint8 [..., hidden] (E4M3 of checkpoint_scale(hidden) times the
    normalised row) and rstd float32 [rows]."""
    if out is None and codes is None and rstd is None and stream is None:
        done = _fast.layer_norm_checkpoint(x, weight, bias, eps)
        if done is not None:
            return done
    rows, hidden, ldx = _pitch(x, "x")
    w, b = _param(weight, hidden, x.dtype, "weight"), _param(bias, hidden, x.dtype, "bias")
    ptype = _param_type(weight, bias, x.dtype)
    at = _Launch(stream, (x, weight, bias, out, codes, rstd))
    out = at.empty(x.shape, x.dtype) if out is None else out
    codes = at.empty(x.shape, torch.uint8) if codes is None else codes
    rstd = at.empty(rows, torch.float32) if rstd is None else rstd
    ldy = _same_rows(out, "out", x.dtype, rows, hidden)
    at.call(_lib.taco_norm_checkpoint, "taco_norm_checkpoint", x.data_ptr(), ldx, rows, hidden,
            DTYPES[x.dtype], w, b, DTYPES[ptype], eps, out.data_ptr(), ldy,
            _codes(codes, rows, hidden), _vector(rstd, rows, "rstd"))
    return out, codes, rstd


def _gradients(at, dy, dx, hidden, ptype, rows, param_grads):
    dx = at.empty(dy.shape, dy.dtype) if dx is None else dx
    lddx = _same_rows(dx, "dx", dy.dtype, rows, hidden)
    if not param_grads:
        return dx, lddx, None, None, None
    dw, db = at.empty(hidden, ptype), at.empty(hidden, ptype)
    return dx, lddx, dw, db, at.workspace(_lib.taco_norm_backward_workspace(rows, hidden))


def layer_norm_backward(dy, x, mean, rstd, weight=None, dx=None, param_grads: bool = True,
                        param_dtype=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias), the last two of
    param_dtype (weight's type; float32 without a weight), or None without
    param_grads.  dx may be dy (in place)."""
    if dx is None and param_grads and param_dtype is None and stream is None:
        done = _fast.layer_norm_backward(dy, x, mean, rstd, weight)
        if done is not None:
            return done
    rows, hidden, lddy = _pitch(dy, "dy")
    ldx = _same_rows(x, "x", dy.dtype, rows, hidden)
    m, r = _vector(mean, rows, "mean"), _vector(rstd, rows, "rstd")
    w, ptype = _backward_param(weight, hidden, dy.dtype, param_dtype)
    at = _Launch(stream, (dy, x, mean, rstd, weight, dx))
    dx, lddx, dw, db, ws = _gradients(at, dy, dx, hidden, ptype, rows, param_grads)
    at.call(_lib.taco_norm_backward, "taco_norm_backward", dy.data_ptr(), lddy, x.data_ptr(), ldx,
            m, r, w, rows, hidden, DTYPES[dy.dtype], DTYPES[ptype], dx.data_ptr(), lddx, _ptr(dw),
            _ptr(db), _ptr(ws), 0 if ws is None else ws.numel())
    return dx, dw, db


def _backward_param(weight, hidden, dtype, param_dtype):
    w = _param(weight, hidden, dtype, "weight")
    ptype = weight.dtype if weight is not None else (param_dtype or torch.float32)
    if param_dtype is not None and param_dtype != ptype:
        raise TypeError(f"param_dtype must be weight's type, {ptype}")
    if ptype != dtype and ptype != torch.float32:
        raise TypeError(f"param_dtype must be {dtype} or torch.float32, got {ptype}")
    return w, ptype


def layer_norm_checkpoint_backward(dy, codes, rstd, weight=None, dx=None,
                                   param_grads: bool = True, param_dtype=None, stream=None):
    """Gradients of layer_norm_checkpoint from its checkpoint: as
    layer_norm_backward, with codes in the place of the saved input."""
    if dx is None and param_grads and param_dtype is None and stream is None:
        done = _fast.layer_norm_checkpoint_backward(dy, codes, rstd, weight)
        if done is not None:
            return done
    rows, hidden, lddy = _pitch(dy, "dy")
    c, r = _codes(codes, rows, hidden), _vector(rstd, rows, "rstd")
    w, ptype = _backward_param(weight, hidden, dy.dtype, param_dtype)
    at = _Launch(stream, (dy, codes, rstd, weight, dx))
    dx, lddx, dw, db, ws = _gradients(at, dy, dx, hidden, ptype, rows, param_grads)
    at.call(_lib.taco_norm_checkpoint_backward, "taco_norm_checkpoint_backward", dy.data_ptr(),
            lddy, c, r, w, rows, hidden, DTYPES[dy.dtype], DTYPES[ptype], dx.data_ptr(), lddx,
            _ptr(dw), _ptr(db), _ptr(ws), 0 if ws is None else ws.numel())
    return dx, dw, db


def checkpoint_weight_grad(dy, codes, weight=None, bias=None, out=None, dtype=None,
                           accumulate: bool = False, bias_grad: bool = True, stream=None):
    """Gradient of a linear layer's weight from the checkpoint of the layer
    norm before it: (dW, db), dW [out_features, hidden] = dy^T y for the
    norm's output y = decode(codes) / S * weight + bias, db [out_features]
    float32 = the rows' sum of dy (None without bias_grad).

    dy: bf16 or fp16 [..., out_features]; codes [..., hidden].  dW is of
    ``dtype`` (dy's type by default, or float32); with ``accumulate`` it is
    added to ``out``, a float32 tensor.  ``out``: [out_features, hidden]."""
    if dtype is None:
        dtype = getattr(dy if out is None else out, "dtype", None)
    # (The fast path writes at once, so it gets no type that is refused below.)
    if bias_grad and stream is None and dtype in (torch.float32, getattr(dy, "dtype", None)):
        done = _fast.checkpoint_weight_grad(dy, codes, weight, bias, out, dtype is torch.float32,
                                            bool(accumulate))
        if done is not None:
            return done
    rows, features, lddy = _pitch(dy, "dy")
    if dy.dtype == torch.float32:
        raise TypeError("dy must be torch.bfloat16 or torch.float16")
    if not isinstance(codes, torch.Tensor) or codes.dim() == 0:
        raise TypeError("codes must be a CUDA/HIP torch tensor [..., hidden]")
    hidden = codes.shape[-1]
    c = _codes(codes, rows, hidden)
    w, b = _param(weight, hidden, dy.dtype, "weight"), _param(bias, hidden, dy.dtype, "bias")
    ptype = _param_type(weight, bias, dy.dtype)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype != dy.dtype and dtype != torch.float32:
        raise TypeError(f"dtype must be {dy.dtype} or torch.float32, got {dtype}")
    if accumulate and dtype != torch.float32:
        raise TypeError("accumulate needs a torch.float32 out")
    at = _Launch(stream, (dy, codes, weight, bias, out))
    out = at.empty((features, hidden), dtype) if out is None else out
    o = _vector(out, features * hidden, "out", dtype)
    if out.shape != (features, hidden):
        raise ValueError(f"out must be [{features}, {hidden}], got {list(out.shape)}")
    db = at.empty(features, torch.float32) if bias_grad else None
    ws = at.workspace(_lib.taco_norm_weight_grad_workspace(dy.data_ptr(), lddy, c, rows, features,
                                                           hidden))
    at.call(_lib.taco_norm_weight_grad, "taco_norm_weight_grad", dy.data_ptr(), lddy, c, rows,
            features, hidden, DTYPES[dy.dtype], w, b, DTYPES[ptype], o, DTYPES[dtype],
            int(accumulate), _ptr(db), _ptr(ws), 0 if ws is None else ws.numel())
    return out, db


def _residual(residual, x, rows, hidden):
    """(device pointer, elements between rows) of a residual like x, or (0, 0)."""
    if residual is None:
        return 0, 0
    ld = _same_rows(residual, "residual", x.dtype, rows, hidden)
    return residual.data_ptr(), ld


def rms_norm(x, weight=None, eps: float = 1e-5, residual=None, out=None, total=None, rstd=None,
             stream=None):
    """Root-mean-square norm of x + residual over the last dimension: (y, total,
    rstd), total = x + residual (None without a residual), rstd float32 [rows], as
    the backward pass takes them.  out and total may be x or residual (in place)."""
    if out is None and total is None and rstd is None and stream is None:
        done = _fast_rms.rms_norm(x, weight, eps, residual)
        if done is not None:
            return done
    rows, hidden, ldx = _pitch(x, "x")
    w = _param(weight, hidden, x.dtype, "weight")
    ptype = _param_type(weight, None, x.dtype)
    r, ldr = _residual(residual, x, rows, hidden)
    if residual is None and total is not None:
        raise ValueError("total needs a residual")
    at = _Launch(stream, (x, weight, residual, out, total, rstd))
    out = at.empty(x.shape, x.dtype) if out is None else out
    if residual is not None and total is None:
        total = at.empty(x.shape, x.dtype)
    rstd = at.empty(rows, torch.float32) if rstd is None else rstd
    ldy = _same_rows(out, "out", x.dtype, rows, hidden)
    ldt = 0 if total is None else _same_rows(total, "total", x.dtype, rows, hidden)
    at.call(_rms.taco_rms_forward, "taco_rms_forward", x.data_ptr(), ldx, r, ldr, rows,
            hidden, DTYPES[x.dtype], w, DTYPES[ptype], eps, out.data_ptr(), ldy, _ptr(total), ldt,
            _vector(rstd, rows, "rstd"))
    return out, total, rstd


def rms_norm_mx(x, weight=None, eps: float = 1e-5, residual=None, total=None, stream=None):
    """rms_norm into 8 bits: (codes, scales, total), codes uint8 [..., hidden] and
    scales uint8 [..., hidden / 32], E4M3 codes of each 32 neighbours over their scale
    2^(byte - 127), as gated.gated_forward_mx takes them.  total may be x or
    residual (in place)."""
    if total is None and stream is None:
        done = _fast_rms.rms_norm_mx(x, weight, eps, residual)
        if done is not None:
            return done
    rows, hidden, ldx = _pitch(x, "x")
    if hidden == 0 or hidden % 32:
        raise ValueError(f"x must hold rows of a multiple of 32, got {list(x.shape)}")
    w = _param(weight, hidden, x.dtype, "weight")
    ptype = _param_type(weight, None, x.dtype)
    r, ldr = _residual(residual, x, rows, hidden)
    if residual is None and total is not None:
        raise ValueError("total needs a residual")
    at = _Launch(stream, (x, weight, residual, total))
    codes = at.empty(x.shape, torch.uint8)
    scales = at.empty((*x.shape[:-1], hidden // 32), torch.uint8)
    if residual is not None and total is None:
        total = at.empty(x.shape, x.dtype)
    ldt = 0 if total is None else _same_rows(total, "total", x.dtype, rows, hidden)
    at.call(_rms.taco_rms_mx, "taco_rms_mx", x.data_ptr(), ldx, r, ldr, rows, hidden,
            DTYPES[x.dtype], w, DTYPES[ptype], eps, codes.data_ptr(), scales.data_ptr(),
            _ptr(total), ldt)
    return codes, scales, total


def rms_norm_backward(dy, x, rstd, weight=None, dtotal=None, dx=None, param_grads: bool = True,
                      param_dtype=None, stream=None):
    """Gradients of rms_norm: (dx, dweight).  x: its total (x without a residual).
    dtotal: the gradient that arrives at total.  dx is the gradient of x and of
    residual alike, and may be dy or dtotal (in place); dweight is of param_dtype
    (weight's type; float32 without a weight), None without param_grads."""
    if dx is None and param_grads and param_dtype is None and stream is None:
        done = _fast_rms.rms_norm_backward(dy, x, rstd, weight, dtotal)
        if done is not None:
            return done
    rows, hidden, lddy = _pitch(dy, "dy")
    ldx = _same_rows(x, "x", dy.dtype, rows, hidden)
    q = _vector(rstd, rows, "rstd")
    w, ptype = _backward_param(weight, hidden, dy.dtype, param_dtype)
    lddt = 0 if dtotal is None else _same_rows(dtotal, "dtotal", dy.dtype, rows, hidden)
    at = _Launch(stream, (dy, x, rstd, weight, dtotal, dx))
    dx = at.empty(dy.shape, dy.dtype) if dx is None else dx
    lddx = _same_rows(dx, "dx", dy.dtype, rows, hidden)
    dw = at.empty(hidden, ptype) if param_grads else None
    ws = (at.workspace(_rms.taco_rms_backward_workspace(rows, hidden)) if param_grads
          else None)
    at.call(_rms.taco_rms_backward, "taco_rms_backward", dy.data_ptr(), lddy,
            x.data_ptr(), ldx, q, _ptr(dtotal), lddt, w, rows, hidden, DTYPES[dy.dtype],
            DTYPES[ptype], dx.data_ptr(), lddx, _ptr(dw), _ptr(ws),
            0 if ws is None else ws.numel())
    return dx, dw


# --------------------------------------------------------------- autograd --

def _even(t):
    """t, or a contiguous copy of it where its rows are not evenly spaced."""
    try:
        _pitch(t, "gradient")
        return t
    except ValueError:
        return t.contiguous()


def _shape(t):
    return None if t is None else t.shape


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm(_even(x), weight, bias, eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.bias_type = None if bias is None else bias.dtype
        ctx.shapes = _shape(weight), _shape(bias)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        want_w, want_b = ctx.needs_input_grad[1:3]
        dx, dw, db = layer_norm_backward(
            _even(dy), _even(x), mean, rstd, weight, param_grads=want_w or want_b,
            param_dtype=ctx.bias_type if weight is None else None)
        return (dx, dw.view(ctx.shapes[0]) if want_w else None,
                db.view(ctx.shapes[1]) if want_b else None, None)


class _Rms(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps):
        x = _even(x)
        y, _, rstd = rms_norm(x, weight, eps)
        ctx.save_for_backward(x, rstd, weight)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = rms_norm_backward(_even(dy), x, rstd, weight, param_grads=need[1])
        return dx if need[0] else None, dw.view(weight.shape) if need[1] else None, None


class _RmsResidual(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, total, rstd = rms_norm(_even(x), weight, eps, residual=_even(residual))
        ctx.save_for_backward(total, rstd, weight)
        ctx.residual_shape = residual.shape
        ctx.set_materialize_grads(False)
        return y, total

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dtotal):
        if dy is None and dtotal is None:    # neither output was given a gradient
            return None, None, None, None
        total, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:                       # y was not used
            # (dtotal may be the caller's, and other gradients' too: handed on as it is,
            # or copied, but not as a view, which autograd would take for new memory)
            dx, dw = dtotal, torch.zeros_like(weight) if need[2] else None
            if need[1] and dx.shape != ctx.residual_shape:
                return dx if need[0] else None, dx.reshape(ctx.residual_shape).clone(), dw, None
        else:
            dtotal = None if dtotal is None else _even(dtotal)
            dx, dw = rms_norm_backward(_even(dy), total, rstd, weight, dtotal=dtotal,
                                       param_grads=need[2])
            dw = dw.view(weight.shape) if need[2] else None
        # (the residual has x's rows, not always its leading dimensions)
        dr = dx if dx.shape == ctx.residual_shape else dx.reshape(ctx.residual_shape)
        return dx if need[0] else None, dr if need[1] else None, dw, None


class _NormLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, linear_weight, linear_bias, eps):
        y, codes, rstd = layer_norm_checkpoint(_even(x), weight, bias, eps)
        ctx.save_for_backward(codes, rstd, weight, bias, linear_weight)
        ctx.linear_bias_type = None if linear_bias is None else linear_bias.dtype
        ctx.type = x.dtype
        return torch.nn.functional.linear(y.to(linear_weight.dtype), linear_weight, linear_bias)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dz):
        codes, rstd, weight, bias, linear_weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        dz = _even(dz)
        grads = [None] * 6
        if need[3] or need[4]:
            # The norm's parameters are of the norm's type, dz of the linear layer's.
            params = [p if p is None or p.dtype == dz.dtype else p.float() for p in (weight, bias)]
            dW, db = checkpoint_weight_grad(dz, codes, *params, dtype=linear_weight.dtype)
            grads[3] = dW if need[3] else None
            if need[4] and ctx.linear_bias_type is not None:
                grads[4] = db.to(ctx.linear_bias_type)
        if any(need[:3]):
            dy = torch.mm(dz.reshape(-1, dz.shape[-1]), linear_weight).view(codes.shape)
            dy = dy.to(ctx.type)
            dx, dw, db = layer_norm_checkpoint_backward(
                dy, codes, rstd, weight, dx=dy, param_grads=need[1] or need[2],
                param_dtype=None if weight is not None or bias is None else bias.dtype)
            grads[:3] = [dx, dw.view(weight.shape) if need[1] else None,
                         db.view(bias.shape) if need[2] else None]
        return tuple(grads)


def norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Differentiable layer norm over the last dimension."""
    return _Norm.apply(x, weight, bias, eps)


def rms(x, weight=None, eps: float = 1e-5, residual=None):
    """Differentiable root-mean-square norm over the last dimension: y, or with
    a residual (y, x + residual).  For its backward pass it keeps the sum (x without a
    residual) and one float32 per row.

    A backward pass may be captured into a graph once no eager graph of the same
    leaves is alive (torch's rule for all of its functions)."""
    if residual is None:
        return _Rms.apply(x, weight, eps)
    return _RmsResidual.apply(x, residual, weight, eps)


def norm_linear(x, weight, bias, linear_weight, linear_bias=None, eps: float = 1e-5):
    """Differentiable ``linear(layer_norm(x))`` for bf16 and fp16 activations.
    For the backward pass it keeps the 8-bit checkpoint of the normalised
    rows and one float32 per row, instead of the norm's input and output.

    x and the linear layer's tensors are of one type.  Under
    ``torch.autocast`` they need not be, and x may be float32: the norm runs
    in x's type and the linear layer in autocast's, as torch's own does there."""
    auto = torch.get_autocast_dtype("cuda") if torch.is_autocast_enabled("cuda") else None
    if auto in (torch.bfloat16, torch.float16):
        for t, name in ((x, "x"), (linear_weight, "linear_weight"), (linear_bias, "linear_bias")):
            if t is not None and t.dtype not in DTYPES:
                raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
        linear_weight = linear_weight.to(auto)
        linear_bias = None if linear_bias is None else linear_bias.to(auto)
    elif x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    elif linear_weight.dtype != x.dtype:
        raise TypeError(f"linear_weight must be {x.dtype}, got {linear_weight.dtype}")
    hidden = x.shape[-1] if x.dim() else 0
    if linear_weight.dim() != 2 or linear_weight.shape[1] != hidden:
        raise ValueError(f"linear_weight must be [out_features, {hidden}], got "
                         f"{list(linear_weight.shape)}")
    if linear_bias is not None and linear_bias.shape != linear_weight.shape[:1]:
        raise ValueError(f"linear_bias must be [{linear_weight.shape[0]}], got "
                         f"{list(linear_bias.shape)}")
    return _NormLinear.apply(x, weight, bias, linear_weight, linear_bias, eps)
