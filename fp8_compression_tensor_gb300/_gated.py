"""Operators of a gated feed-forward block behind an RMS norm, next to the
training operators of _training.py (include/taco.h):

    r = rmsnorm(x, weight, residual=None, checkpoint=True)           # r.y, r.rstd, r.summed, r.packed
    g = rmsnorm_backward(dy, r.rstd, weight, packed=r.packed)        # g.dx, g.dweight
    r = gated_linear(x, weight, checkpoint=True)                     # r.y, r.packed
    g = gated_linear_backward(dy, r.packed, weight)                  # g.dz, g.dx, g.dbias, g.y
    dw = weight_grad(g.dz, packed, hidden)                           # the projections' weights, X kept as records (bf16)

Argument marshalling only.  No call records an autograd graph: the forward and
backward calls are for a torch.autograd.Function, as in
examples/gated_block_8bit.py.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import _training
from ._binding import _check, _raw_stream
from ._training import (DTYPES, _address, _code, _f32, _first, _i32, _i64, _packed, _packer, _param_type, _ptr, _record_bytes,
                        _run, _tensor, _workspace_bytes)

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}   # taco_activation_t


class _RmsNormArgs(ctypes.Structure):
    _fields_ = [("x", _ptr), ("residual", _ptr), ("weight", _ptr), ("y", _ptr), ("summed", _ptr), ("rstd", _ptr),
                ("packed", _ptr), ("packed_y", _ptr), ("rows", _i64), ("hidden", _i64), ("eps", _f32), ("dtype", _i32),
                ("param_dtype", _i32), ("block", _i32), ("code", _i32)]


class _RmsNormBackwardArgs(ctypes.Structure):
    _fields_ = [("dy", _ptr), ("x", _ptr), ("rstd", _ptr), ("packed", _ptr), ("weight", _ptr), ("dsummed", _ptr),
                ("dx", _ptr), ("dweight", _ptr), ("workspace", _ptr), ("workspace_bytes", _i64), ("rows", _i64),
                ("hidden", _i64), ("dtype", _i32), ("param_dtype", _i32), ("block", _i32), ("code", _i32)]


class _GatedLinearArgs(ctypes.Structure):
    _fields_ = [("x", _ptr), ("weight", _ptr), ("bias", _ptr), ("y", _ptr), ("packed", _ptr), ("workspace", _ptr),
                ("workspace_bytes", _i64), ("rows", _i64), ("inner", _i64), ("hidden", _i64), ("dtype", _i32),
                ("param_dtype", _i32), ("activation", _i32), ("block", _i32), ("code", _i32)]


class _GatedLinearBackwardArgs(ctypes.Structure):
    _fields_ = [("dy", _ptr), ("packed", _ptr), ("weight", _ptr), ("dz", _ptr), ("dx", _ptr), ("y", _ptr),
                ("dbias", _ptr), ("workspace", _ptr), ("workspace_bytes", _i64), ("rows", _i64), ("inner", _i64),
                ("hidden", _i64), ("dtype", _i32), ("param_dtype", _i32), ("activation", _i32), ("block", _i32),
                ("code", _i32)]


_CALLS = {"taco_rmsnorm": _RmsNormArgs, "taco_rmsnorm_backward": _RmsNormBackwardArgs, "taco_gated_linear": _GatedLinearArgs,
          "taco_gated_linear_backward": _GatedLinearBackwardArgs}
_pack_rmsnorm, _pack_rmsnorm_backward = _packer(_RmsNormArgs), _packer(_RmsNormBackwardArgs)
_pack_gated, _pack_gated_backward = _packer(_GatedLinearArgs), _packer(_GatedLinearBackwardArgs)

_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = _training._library()
        for name in _CALLS:
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [_ptr, _ptr], _i32
        lib.taco_rmsnorm_backward_workspace.argtypes = [_i64, _i64]
        lib.taco_gated_linear_workspace.argtypes = lib.taco_gated_linear_backward_workspace.argtypes = [_i64, _i64, _i64]
        for name in ("taco_rmsnorm_backward_workspace", "taco_gated_linear_workspace", "taco_gated_linear_backward_workspace"):
            getattr(lib, name).restype = _i64
        _lib = lib
    return _lib


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(device: int, stream, call, *args):
    """call(handle, *args) on the device and the stream (_training._run).  On the
    current ones it is called directly: a closure and the look for a device
    cost two of the fifteen microseconds of a small call."""
    if stream is None and _raw_stream is not None and device == _current_device():
        return call(_raw_stream(device), *args)
    return _run(device, stream, lambda handle: call(handle, *args))


class RmsNorm(NamedTuple):
    y: torch.Tensor
    rstd: torch.Tensor
    summed: Optional[torch.Tensor]
    packed: Optional[torch.Tensor]


class RmsNormGrads(NamedTuple):
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]


class GatedLinear(NamedTuple):
    y: torch.Tensor
    packed: Optional[torch.Tensor]


class GatedLinearGrads(NamedTuple):
    dz: torch.Tensor
    dx: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]
    y: Optional[torch.Tensor]


def rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
            residual: Optional[torch.Tensor] = None, checkpoint: bool = False, packed_y: bool = False, block: int = 128,
            code="e4m3", stream=None) -> RmsNorm:
    """Root-mean-square norm over the last dimension of x (bf16, f16 or f32), or
    of x + residual (rounded to x's type and returned as `summed`).  rstd is
    float32, one per row (NaN for rows of no elements).  With packed_y, y is a
    uint8 tensor of 8-bit records (made from the float32 values; decompress(y,
    rows, hidden, block, variant="ds_only", code=code) gives them).  With
    checkpoint, `packed` holds the normalised rows (before the weight) as
    records."""
    kind, rows, hidden = _first(x, "x")
    device, shape = x.get_device(), x.shape
    pdtype = _param_type(weight, "weight")
    pr = _tensor(residual, "residual", device, x.dtype, shape)
    pw = _tensor(weight, "weight", device, pdtype, (hidden,))
    nbytes = _record_bytes(rows, hidden, block) if checkpoint or packed_y else 0
    rc, result = _launch(device, stream, _rmsnorm, x, pw, eps, residual is not None, pr, checkpoint, packed_y, nbytes, rows,
                         hidden, kind, DTYPES[pdtype], block, _code(code))
    if rc:
        _check(rc, "taco_rmsnorm")
    return result


def _rmsnorm(handle, x, weight, eps, add, residual, checkpoint, packed_y, nbytes, rows, hidden, kind, pkind, block, code):
    device = x.device
    y = torch.empty(nbytes, dtype=torch.uint8, device=device) if packed_y else torch.empty_like(x)
    summed = torch.empty_like(x) if add else None
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    if hidden == 0:   # no element to average: 0 / 0 (the library launches nothing)
        rstd.fill_(math.nan)
    packed = torch.empty(nbytes, dtype=torch.uint8, device=device) if checkpoint else None
    py = y.data_ptr()
    rc = _library().taco_rmsnorm(
        _pack_rmsnorm(x.data_ptr(), residual, weight, 0 if packed_y else py, _address(summed), rstd.data_ptr(), _address(packed),
                      py if packed_y else 0, rows, hidden, eps, kind, pkind, block, code), handle)
    return rc, RmsNorm(y, rstd, summed, packed)


def rmsnorm_backward(dy: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                     x: Optional[torch.Tensor] = None, packed: Optional[torch.Tensor] = None,
                     dsummed: Optional[torch.Tensor] = None, block: int = 128, code="e4m3", stream=None) -> RmsNormGrads:
    """Gradients of rmsnorm from either x, what was normalised (`summed` where
    there was a residual), or the records `packed`.  dsummed, the gradient that
    reaches `summed` from elsewhere, is added to dx.  dweight is in weight's
    type, and None without a weight."""
    if (x is None) == (packed is None):
        raise ValueError("give either x or packed")
    kind, rows, hidden = _first(dy, "dy")
    device, shape = dy.get_device(), dy.shape
    pdtype = _param_type(weight, "weight")
    prstd = _tensor(rstd, "rstd", device, torch.float32, shape[:-1])
    px = _tensor(x, "x", device, dy.dtype, shape)
    ppacked = 0 if packed is None else _packed(packed, rows, hidden, block, device)
    pw = _tensor(weight, "weight", device, pdtype, (hidden,))
    pds = _tensor(dsummed, "dsummed", device, dy.dtype, shape)
    rc, result = _launch(device, stream, _rmsnorm_backward, dy, px, prstd, ppacked, weight, pw, pds, rows, hidden, kind,
                         DTYPES[pdtype], block, _code(code))
    if rc:
        _check(rc, "taco_rmsnorm_backward")
    return result


def _rmsnorm_backward(handle, dy, x, rstd, packed, weight, pweight, dsummed, rows, hidden, kind, pkind, block, code):
    lib = _library()
    dx = torch.empty_like(dy)
    dweight = ws = None
    nbytes = 0
    if weight is not None:
        dweight = torch.empty_like(weight)
        nbytes = _workspace_bytes("taco_rmsnorm_backward_workspace", rows, hidden)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
    rc = lib.taco_rmsnorm_backward(
        _pack_rmsnorm_backward(dy.data_ptr(), x, rstd, packed, pweight, dsummed, dx.data_ptr(), _address(dweight), _address(ws),
                               nbytes, rows, hidden, kind, pkind, block, code), handle)
    return rc, RmsNormGrads(dx, dweight)


def _activation(name: str) -> int:
    kind = ACTIVATIONS.get(name)
    if kind is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return kind


def _half(t, name: str):
    """_first for tensors of 16 bits."""
    made = _first(t, name)
    if made[0] == 2:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return made


def _halves(features: int, name: str) -> int:
    if features % 2:
        raise ValueError(f"{name} must have the gate's rows and as many of the up projection, has {features}")
    return features // 2


def gated_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: str = "silu",
                 checkpoint: bool = False, block: int = 128, code="e4m3", stream=None) -> GatedLinear:
    """act(x Wg^T + bg) * (x Wu^T + bu) for x [..., hidden] (bf16 or f16, hidden
    up to 2^24) and weight [2 inner, hidden] of x's type, the gate's rows Wg before the up
    projection's Wu; bias [2 inner].  The activation is "silu", "gelu" or
    "gelu_tanh".  With checkpoint, `packed` holds both projections' float32
    values [..., 2 inner] as records (blocks 32, 64 and 128)."""
    act = _activation(activation)
    kind, rows, hidden = _half(x, "x")
    device = x.get_device()
    _first(weight, "weight")
    inner = _halves(weight.shape[0], "weight")
    pw = _tensor(weight, "weight", device, x.dtype, (2 * inner, hidden))
    pdtype = _param_type(bias, "bias")
    pb = _tensor(bias, "bias", device, pdtype, (2 * inner,))
    if hidden == 0:
        raise ValueError("x must have at least one column")
    nbytes = _record_bytes(rows, 2 * inner, block) if checkpoint else 0
    rc, result = _launch(device, stream, _gated_linear, x, pw, pb, checkpoint, nbytes, rows, inner, hidden, kind, DTYPES[pdtype],
                         act, block, _code(code))
    if rc:
        _check(rc, "taco_gated_linear")
    return result


def _gated_linear(handle, x, weight, bias, checkpoint, nbytes, rows, inner, hidden, kind, pkind, activation, block, code):
    lib, device = _library(), x.device
    y = torch.empty((*x.shape[:-1], inner), dtype=x.dtype, device=device)
    packed = torch.empty(nbytes, dtype=torch.uint8, device=device) if checkpoint else None
    wbytes = _workspace_bytes("taco_gated_linear_workspace", rows, inner, hidden)
    ws = torch.empty(wbytes, dtype=torch.uint8, device=device) if wbytes > 0 else None
    rc = lib.taco_gated_linear(
        _pack_gated(x.data_ptr(), weight, bias, y.data_ptr(), _address(packed), _address(ws), wbytes, rows, inner, hidden, kind,
                    pkind, activation, block, code), handle)
    return rc, GatedLinear(y, packed)


def gated_linear_backward(dy: torch.Tensor, packed: torch.Tensor, weight: Optional[torch.Tensor] = None,
                          activation: str = "silu", bias_dtype: Optional[torch.dtype] = None, recompute: bool = False,
                          block: int = 128, code="e4m3", stream=None) -> GatedLinearGrads:
    """Gradients of gated_linear from its records, for dy [..., inner]: dz
    [..., 2 inner], the projections' gradient in dy's type; with weight the
    input's gradient dx = dz weight; with bias_dtype the sum of dz over rows in
    that type; with recompute the output y again, for the next layer's weight
    gradient.  The weight's own gradient is weight_grad(dz, records of x,
    hidden), which takes bf16 alone: for f16 it is a product of dz with x as it
    was, outside this package."""
    act = _activation(activation)
    if bias_dtype is not None and bias_dtype not in DTYPES:
        raise TypeError(f"bias_dtype must be bfloat16, float16 or float32, got {bias_dtype}")
    kind, rows, inner = _half(dy, "dy")
    device = dy.get_device()
    if inner == 0:
        raise ValueError("dy must have at least one column")
    ppacked = _packed(packed, rows, 2 * inner, block, device)
    hidden = pw = 0
    if weight is not None:
        _, _, hidden = _first(weight, "weight")
        if hidden == 0:
            raise ValueError("weight must have at least one column")
        pw = _tensor(weight, "weight", device, dy.dtype, (2 * inner, hidden))
    rc, result = _launch(device, stream, _gated_linear_backward, dy, ppacked, weight is not None, pw, bias_dtype, recompute, rows,
                         inner, hidden, kind, act, block, _code(code))
    if rc:
        _check(rc, "taco_gated_linear_backward")
    return result


def _gated_linear_backward(handle, dy, packed, input_grad, weight, bias_dtype, recompute, rows, inner, hidden, kind, activation,
                           block, code):
    lib, device, lead = _library(), dy.device, dy.shape[:-1]
    dz = torch.empty((*lead, 2 * inner), dtype=dy.dtype, device=device)
    dx = torch.empty((*lead, hidden), dtype=dy.dtype, device=device) if input_grad else None
    y = torch.empty_like(dy) if recompute else None
    dbias = torch.empty(2 * inner, dtype=bias_dtype, device=device) if bias_dtype is not None else None
    nbytes = _workspace_bytes("taco_gated_linear_backward_workspace", rows, inner, hidden)
    if bias_dtype is None:   # without the bias gradient's part
        nbytes -= _workspace_bytes("taco_gated_linear_backward_workspace", rows, inner, 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None
    rc = lib.taco_gated_linear_backward(
        _pack_gated_backward(dy.data_ptr(), packed, weight, dz.data_ptr(), _address(dx), _address(y), _address(dbias), _address(ws),
                             nbytes, rows, inner, hidden, kind, DTYPES[bias_dtype or torch.float32], activation, block, code),
        handle)
    return rc, GatedLinearGrads(dz, dx, dbias, y)
