"""Binding of libtaco_gated (include/taco_gated.h): the first half of the gated
feed-forward block -- both projections, the activation and the product in one
kernel -- with its backward pass, and its forward pass on 8-bit codes with
block scales.

    G = X Wg^T,  U = X Wu^T,  A = act(G) U        (act: silu, gelu or gelu_tanh)

Three layers:

* ``taco_gated_*``: the C ABI with the same names and arguments (device
  pointers and stream handles as ints).
* ``gated_forward``, ``gated_backward``, ``gated_forward_mx``, ``mx_encode``: the
  same calls on torch tensors, allocating outputs and workspaces and launching
  on torch's current stream.
* ``gated``: the differentiable block made of them.

X and the weights are bf16 or fp16 tensors whose rows are contiguous and
evenly spaced; X is [..., hidden], the weights [features, hidden] (two halves of
one [2 features, hidden] tensor are fine).  ``norm.rms_norm`` gives X, and
``norm.rms_norm_mx`` gives it in the 8-bit form.
"""
from __future__ import annotations

import ctypes
import os

import torch
from torch.autograd import forward_ad

from . import TacoError  # noqa: F401  (torch's HIP runtime is loaded first)
from .norm import DTYPES, _check, _device_tensor, _even, _Launch, _pitch, _ptr, _same_rows

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtaco_gated.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libtaco_gated.so is not built ({LIB_PATH} missing); run "
        "`python gradients_taco_compress_amd/build.py` (there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

# The usual calls, without the interpreter between them and the C ABI: each
# function returns None for what is not usual (the code below then takes over, and
# words the errors).
try:
    from . import _gated_torch as _fast
except ImportError as e:
    raise ImportError(f"the torch module of libtaco_gated is not built ({e}); run "
                      "`python gradients_taco_compress_amd/build.py`") from e

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_STATUS = ctypes.c_int
_SIGNATURES = {
    "taco_gated_forward_workspace": ([_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64], _I64),
    "taco_gated_forward": ([_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _I32, _I32, _P, _I64,
                            _P, _P, _I64, _P, _I64, _P], _STATUS),
    "taco_gated_backward_workspace": ([_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _I32, _I32],
                                      _I64),
    "taco_gated_backward": ([_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _I64, _I64,
                             _I64, _I32, _I32, _P, _I64, _P, _P, _P, _I64, _P], _STATUS),
    "taco_gated_forward_mx_workspace": ([_I64, _I64, _I64], _I64),
    "taco_gated_forward_mx": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _P, _I64, _P,
                               _I64, _P], _STATUS),
    "taco_gated_mx_encode": ([_P, _I64, _I64, _I64, _I32, _P, _P, _P], _STATUS),
}
#: Symbols the library exports (checked against include/taco_gated.h).
EXPORTS = tuple(_SIGNATURES)
for _name, (_args, _res) in _SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes, _fn.restype = _args, _res
    globals()[_name] = _fn

#: taco_gated_activation of the names.
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
#: Neighbours of a row that share a scale.
MX_BLOCK = 32


# ------------------------------------------------------------- arguments --

def _activation(name):
    if not isinstance(name, str) or name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _type(t, name):
    _device_tensor(t, name)
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return t.dtype


def _weight(t, name, dtype, hidden, features=None):
    """(features, elements between rows) of a weight [features, hidden]."""
    _device_tensor(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] != hidden or (features is not None and t.shape[0] != features):
        want = "features" if features is None else features
        raise ValueError(f"{name} must be [{want}, {hidden}], got {list(t.shape)}")
    return t.shape[0], _pitch(t, name, dtype)[2]


def _mx(pair, name):
    """(codes, scales, rows, hidden) of a pair of contiguous byte tensors."""
    if not isinstance(pair, (tuple, list)) or len(pair) != 2:
        raise TypeError(f"{name} must be a pair (codes, scales)")
    codes, scales = pair
    for t, what in ((codes, "codes"), (scales, "scales")):
        _device_tensor(t, f"{name} {what}")
        if t.dtype != torch.uint8:
            raise TypeError(f"{name} {what} must be torch.uint8, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} {what} must be contiguous")
    hidden = codes.shape[-1] if codes.dim() else 0
    if hidden == 0 or hidden % MX_BLOCK:
        raise ValueError(f"{name} codes must hold rows of a multiple of {MX_BLOCK}, got "
                         f"{list(codes.shape)}")
    if scales.shape != (*codes.shape[:-1], hidden // MX_BLOCK):
        raise ValueError(f"{name} scales must be {[*codes.shape[:-1], hidden // MX_BLOCK]}, got "
                         f"{list(scales.shape)}")
    return codes, scales, codes.numel() // hidden, hidden


def _size(ws):
    return 0 if ws is None else ws.numel()


# -------------------------------------------------------------- operators --

def gated_forward(x, gate_weight, up_weight, activation: str = "silu", save: bool = False,
                  out=None, stream=None):
    """act(x gate_weight^T) * (x up_weight^T): [..., features].  With ``save``:
    (a, gate, up), gate and up the two projections as gated_backward takes them."""
    if out is None and stream is None:
        done = _fast.gated_forward(x, gate_weight, up_weight, ACTIVATIONS.get(activation), bool(save))
        if done is not None:
            return done
    dtype, act = _type(x, "x"), _activation(activation)
    rows, hidden, ldx = _pitch(x, "x")
    features, ldg = _weight(gate_weight, "gate_weight", dtype, hidden)
    _, ldu = _weight(up_weight, "up_weight", dtype, hidden, features)
    at = _Launch(stream, (x, gate_weight, up_weight, out))
    shape = (*x.shape[:-1], features)
    out = at.empty(shape, dtype) if out is None else out
    if out.shape != shape:
        raise ValueError(f"out must be {list(shape)}, got {list(out.shape)}")
    lda = _same_rows(out, "out", dtype, rows, features)
    gate, up = (at.empty(shape, dtype), at.empty(shape, dtype)) if save else (None, None)
    args = (x.data_ptr(), ldx, gate_weight.data_ptr(), ldg, up_weight.data_ptr(), ldu, rows,
            hidden, features)
    ws = at.workspace(_lib.taco_gated_forward_workspace(*args))
    at.call(_lib.taco_gated_forward, "taco_gated_forward", *args, DTYPES[dtype], act,
            out.data_ptr(), lda, _ptr(gate), _ptr(up), features, _ptr(ws), _size(ws))
    return (out, gate, up) if save else out


def gated_backward(da, x, gate, up, gate_weight, up_weight, activation: str = "silu",
                   input_grad: bool = True, weight_grads: bool = True, stream=None):
    """Gradients of gated_forward from its saved projections: (dx,
    dgate_weight, dup_weight), None for those that are not asked for."""
    if input_grad and weight_grads and stream is None:
        done = _fast.gated_backward(da, x, gate, up, gate_weight, up_weight,
                                    ACTIVATIONS.get(activation))
        if done is not None:
            return done
    dtype, act = _type(da, "da"), _activation(activation)
    rows, features, ldda = _pitch(da, "da")
    ldgu = _same_rows(gate, "gate", dtype, rows, features)
    ldup = _same_rows(up, "up", dtype, rows, features)
    hidden = x.shape[-1] if isinstance(x, torch.Tensor) and x.dim() else 0
    ldx = _same_rows(x, "x", dtype, rows, hidden)
    _, ldg = _weight(gate_weight, "gate_weight", dtype, hidden, features)
    _, ldu = _weight(up_weight, "up_weight", dtype, hidden, features)
    at = _Launch(stream, (da, x, gate, up, gate_weight, up_weight))
    if ldup != ldgu:
        with torch.cuda.stream(at.stream):     # (in the order of that stream's work)
            gate, up, ldgu = gate.contiguous(), up.contiguous(), features
    dx = at.empty(x.shape, dtype) if input_grad else None
    dg, du = ((at.empty((features, hidden), dtype), at.empty((features, hidden), dtype))
              if weight_grads else (None, None))
    weights = (gate_weight.data_ptr(), ldg, up_weight.data_ptr(), ldu, rows, hidden, features)
    ws = at.workspace(_lib.taco_gated_backward_workspace(x.data_ptr(), ldx, *weights, input_grad,
                                                         weight_grads))
    at.call(_lib.taco_gated_backward, "taco_gated_backward", da.data_ptr(), ldda, x.data_ptr(), ldx,
            gate.data_ptr(), up.data_ptr(), ldgu, *weights, DTYPES[dtype], act, _ptr(dx), hidden,
            _ptr(dg), _ptr(du), _ptr(ws), _size(ws))
    return dx, dg, du


def mx_encode(x, stream=None):
    """(codes, scales) of rows [..., hidden], hidden a multiple of 32: bytes, E4M3
    codes of each 32 neighbours over their scale 2^(byte - 127)."""
    rows, hidden, ldx = _pitch(x, "x")
    if hidden == 0 or hidden % MX_BLOCK:
        raise ValueError(f"x must hold rows of a multiple of {MX_BLOCK}, got {list(x.shape)}")
    at = _Launch(stream, (x,))
    codes = at.empty(x.shape, torch.uint8)
    scales = at.empty((*x.shape[:-1], hidden // MX_BLOCK), torch.uint8)
    at.call(_lib.taco_gated_mx_encode, "taco_gated_mx_encode", x.data_ptr(), ldx, rows, hidden,
            DTYPES[x.dtype], codes.data_ptr(), scales.data_ptr())
    return codes, scales


def gated_forward_mx(x, gate_weight, up_weight, activation: str = "silu", dtype=torch.bfloat16,
                     out=None, stream=None):
    """gated_forward on 8-bit operands: x, gate_weight and up_weight are pairs
    (codes, scales) as norm.rms_norm_mx and mx_encode return them.  The result is
    of ``dtype`` (bf16 or fp16)."""
    if out is None and stream is None and dtype in (torch.bfloat16, torch.float16):
        done = _fast.gated_forward_mx(x, gate_weight, up_weight, ACTIVATIONS.get(activation),
                                      dtype is torch.float16)
        if done is not None:
            return done
    act = _activation(activation)
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    xc, xs, rows, hidden = _mx(x, "x")
    gc, gs, features, gh = _mx(gate_weight, "gate_weight")
    uc, us, _, _ = _mx(up_weight, "up_weight")
    if gc.dim() != 2 or gh != hidden:
        raise ValueError(f"gate_weight codes must be [features, {hidden}], got {list(gc.shape)}")
    if uc.shape != gc.shape:
        raise ValueError(f"up_weight codes must be {list(gc.shape)}, got {list(uc.shape)}")
    at = _Launch(stream, (xc, xs, gc, gs, uc, us, out))
    shape = (*xc.shape[:-1], features)
    out = at.empty(shape, dtype) if out is None else out
    if out.shape != shape:
        raise ValueError(f"out must be {list(shape)}, got {list(out.shape)}")
    lda = _same_rows(out, "out", dtype, rows, features)
    ws = at.workspace(_lib.taco_gated_forward_mx_workspace(rows, hidden, features))
    at.call(_lib.taco_gated_forward_mx, "taco_gated_forward_mx", xc.data_ptr(), xs.data_ptr(),
            gc.data_ptr(), gs.data_ptr(), uc.data_ptr(), us.data_ptr(), rows, hidden, features,
            DTYPES[dtype], act, out.data_ptr(), lda, _ptr(ws), _size(ws))
    return out


# --------------------------------------------------------------- autograd --

class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate_weight, up_weight, activation):
        x, gate_weight, up_weight = _even(x), _even(gate_weight), _even(up_weight)
        ctx.activation = activation
        if not any(ctx.needs_input_grad):
            return gated_forward(x, gate_weight, up_weight, activation)
        a, gate, up = gated_forward(x, gate_weight, up_weight, activation, save=True)
        ctx.save_for_backward(x, gate, up, gate_weight, up_weight)
        return a

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, da):
        x, gate, up, gate_weight, up_weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dg, du = gated_backward(_even(da), x, gate, up, gate_weight, up_weight,
                                    ctx.activation, input_grad=need[0],
                                    weight_grads=need[1] or need[2])
        return dx, dg if need[1] else None, du if need[2] else None, None


def _tangents(*tensors):
    """Whether a tensor carries a tangent (forward-mode differentiation, which
    torch.no_grad does not turn off, and which autograd refuses for the block)."""
    if getattr(forward_ad, "_current_level", 0) < 0:       # none is open: the usual case
        return False
    return any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None
               for t in tensors)


def gated(x, gate_weight, up_weight, activation: str = "silu"):
    """Differentiable ``act(x gate_weight^T) * (x up_weight^T)``.  It keeps x and
    both projections for its backward pass, nothing without gradients.  It has no
    forward-mode derivative: a tangent is refused.

    The tensors are of one type, bf16 or fp16.  Under ``torch.autocast`` they need
    not be: they are cast to autocast's type, as torch's own linear layer does there,
    and gradients are in the leaves' types.

    A backward pass may be captured into a graph once no eager graph of the same
    leaves is alive (torch's rule for all of its functions)."""
    auto = torch.get_autocast_dtype("cuda") if torch.is_autocast_enabled("cuda") else None
    if auto in (torch.bfloat16, torch.float16):
        for t, name in ((x, "x"), (gate_weight, "gate_weight"), (up_weight, "up_weight")):
            _device_tensor(t, name)
            if t.dtype not in DTYPES:
                raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
        x, gate_weight, up_weight = (t.to(auto) for t in (x, gate_weight, up_weight))
    if not torch.is_grad_enabled() and not _tangents(x, gate_weight, up_weight):
        return gated_forward(_even(x), _even(gate_weight), _even(up_weight), activation)
    return _Gated.apply(x, gate_weight, up_weight, activation)
