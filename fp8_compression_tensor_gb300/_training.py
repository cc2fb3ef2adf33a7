"""Training operators around the compressed tensors: layer norm, GELU, 8-bit
checkpoints of activations and the gradients that read them (the "Training
operators" of include/taco.h).

    r = layernorm(x, weight, bias, residual=None, checkpoint=True)   # r.y, r.mean, r.rstd, r.summed, r.packed
    g = layernorm_backward(dy, r.rstd, weight, packed=r.packed)      # g.dx, g.dweight, g.dbias
    r = gelu(x, bias)                                                # r.y, r.packed
    g = gelu_backward(dy, r.packed, bias_dtype=torch.float32)        # g.dx, g.dbias, g.y
    dw = weight_grad(dy, packed, hidden)                             # dy^T X, X kept as records

A checkpoint is a uint8 tensor of compressed_bytes(rows, hidden, block) bytes
of DS-only records with power-of-two scales;
decompress(packed, rows, hidden, block, variant="ds_only") gives its values.
Argument marshalling only, like _binding.  No call records an autograd graph:
the forward and backward calls are for a torch.autograd.Function, as in
examples/mlp_block_8bit.py.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
from typing import NamedTuple, Optional

import torch

from ._binding import CODES, _check, _raw_stream, compressed_bytes, load_library

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_i64, _i32, _f32, _ptr = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p


class _LayerNormArgs(ctypes.Structure):
    _fields_ = [("x", _ptr), ("residual", _ptr), ("weight", _ptr), ("bias", _ptr), ("y", _ptr), ("summed", _ptr),
                ("mean", _ptr), ("rstd", _ptr), ("packed", _ptr), ("rows", _i64), ("hidden", _i64), ("eps", _f32),
                ("dtype", _i32), ("param_dtype", _i32), ("block", _i32), ("code", _i32)]


class _LayerNormBackwardArgs(ctypes.Structure):
    _fields_ = [("dy", _ptr), ("x", _ptr), ("mean", _ptr), ("rstd", _ptr), ("packed", _ptr), ("weight", _ptr),
                ("dsummed", _ptr), ("dx", _ptr), ("dweight", _ptr), ("dbias", _ptr), ("workspace", _ptr),
                ("workspace_bytes", _i64), ("rows", _i64), ("hidden", _i64), ("dtype", _i32), ("param_dtype", _i32),
                ("block", _i32), ("code", _i32)]


class _GeluArgs(ctypes.Structure):
    _fields_ = [("x", _ptr), ("bias", _ptr), ("y", _ptr), ("packed", _ptr), ("rows", _i64), ("hidden", _i64),
                ("dtype", _i32), ("param_dtype", _i32), ("tanh_form", _i32), ("block", _i32), ("code", _i32)]


class _GeluBackwardArgs(ctypes.Structure):
    _fields_ = [("dy", _ptr), ("packed", _ptr), ("dx", _ptr), ("y", _ptr), ("dbias", _ptr), ("workspace", _ptr),
                ("workspace_bytes", _i64), ("rows", _i64), ("hidden", _i64), ("dtype", _i32), ("param_dtype", _i32),
                ("tanh_form", _i32), ("block", _i32), ("code", _i32)]


class _WeightGradArgs(ctypes.Structure):
    _fields_ = [("dy", _ptr), ("packed", _ptr), ("dweight", _ptr), ("scale", _ptr), ("shift", _ptr), ("dy_sum", _ptr),
                ("workspace", _ptr), ("workspace_bytes", _i64), ("rows", _i64), ("out", _i64), ("hidden", _i64),
                ("dtype", _i32), ("param_dtype", _i32), ("accumulate", _i32), ("block", _i32), ("code", _i32)]


_CALLS = {"taco_layernorm": _LayerNormArgs, "taco_layernorm_backward": _LayerNormBackwardArgs, "taco_gelu": _GeluArgs,
          "taco_gelu_backward": _GeluBackwardArgs, "taco_weight_grad": _WeightGradArgs}


def _packer(kind):
    """struct.Struct of an argument block: packing a short bytes object costs a
    fraction of filling a ctypes structure, which counts in small calls."""
    code = {_ptr: "P", _i64: "q", _i32: "i", _f32: "f"}
    s = struct.Struct("@" + "".join(code[t] for _, t in kind._fields_) + "0q")
    assert s.size == ctypes.sizeof(kind)
    return s.pack


_pack_layernorm, _pack_layernorm_backward = _packer(_LayerNormArgs), _packer(_LayerNormBackwardArgs)
_pack_gelu, _pack_gelu_backward, _pack_weight_grad = _packer(_GeluArgs), _packer(_GeluBackwardArgs), _packer(_WeightGradArgs)

_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = load_library()
        for name in _CALLS:
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [_ptr, _ptr], _i32
        for name in ("taco_layernorm_backward_workspace", "taco_gelu_backward_workspace"):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [_i64, _i64], _i64
        lib.taco_weight_grad_workspace.argtypes, lib.taco_weight_grad_workspace.restype = [_i64, _i64, _i64], _i64
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=512)
def _record_bytes(rows: int, hidden: int, block: int) -> int:
    return compressed_bytes(rows, hidden, block)


@functools.lru_cache(maxsize=512)
def _workspace_bytes(query: str, *sizes: int) -> int:
    """The library's answer for these sizes; 0 for sizes that the call itself refuses."""
    return max(getattr(_library(), query)(*sizes), 0)


class LayerNorm(NamedTuple):
    y: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    summed: Optional[torch.Tensor]
    packed: Optional[torch.Tensor]


class LayerNormGrads(NamedTuple):
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class Gelu(NamedTuple):
    y: torch.Tensor
    packed: Optional[torch.Tensor]


class GeluGrads(NamedTuple):
    dx: torch.Tensor
    dbias: Optional[torch.Tensor]
    y: Optional[torch.Tensor]


def _code(code) -> int:
    return CODES[code] if isinstance(code, str) else int(code)


def _first(x, name: str):
    """Checks the leading tensor of a call: its dtype's number, rows, hidden."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    kind = DTYPES.get(x.dtype)
    if kind is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    shape = x.shape
    if len(shape) == 2:
        return kind, shape[0], shape[1]
    if not shape:
        raise ValueError("tensor must have at least one dimension")
    return kind, math.prod(shape[:-1]), shape[-1]


def _tensor(t, name: str, device: int, dtype, shape) -> int:
    """Checks one more tensor and returns its address (0 for None)."""
    if t is None:
        return 0
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, not on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    return t.data_ptr()


def _param_type(t, name: str):
    if t is None:
        return torch.float32
    if not isinstance(t, torch.Tensor) or t.dtype not in DTYPES:
        raise TypeError(f"{name} must be a bfloat16, float16 or float32 CUDA tensor")
    return t.dtype


def _packed(packed, rows: int, hidden: int, block: int, device: int) -> int:
    return _tensor(packed, "packed", device, torch.uint8, (_record_bytes(rows, hidden, block),))


def _run(device: int, stream, call):
    """Runs call(handle) on the device and the stream.  Tensors allocated in the
    call belong to that stream, so one that is freed while the kernels still run
    (a workspace) is reused behind them only."""
    if stream is None and device == torch.cuda.current_device():
        return call(_raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream)
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream(device).cuda_stream)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _address(t) -> int:
    return 0 if t is None else t.data_ptr()


def layernorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              eps: float = 1e-5, residual: Optional[torch.Tensor] = None, checkpoint: bool = False, block: int = 128,
              code="e4m3", stream=None) -> LayerNorm:
    """Layer norm over the last dimension of x (bf16, f16 or f32), or of
    x + residual (rounded to x's type and returned as `summed`).  weight and
    bias share one type.  mean and rstd are float32, one per row (NaN for rows
    of no elements).  With checkpoint, `packed` holds the normalised rows (before weight and bias) as
    8-bit records."""
    kind, rows, hidden = _first(x, "x")
    device, shape, width = x.get_device(), x.shape, (hidden,)
    pdtype = _param_type(weight if weight is not None else bias, "weight")
    pr = _tensor(residual, "residual", device, x.dtype, shape)
    pw = _tensor(weight, "weight", device, pdtype, width)
    pb = _tensor(bias, "bias", device, pdtype, width)
    nbytes = _record_bytes(rows, hidden, block) if checkpoint else 0

    def call(handle):
        y = torch.empty_like(x)
        summed = torch.empty_like(x) if residual is not None else None
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        if hidden == 0:   # no element to average: 0 / 0 (the library launches nothing)
            for t in (mean, rstd):
                t.fill_(math.nan)
        packed = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if checkpoint else None
        rc = _library().taco_layernorm(
            _pack_layernorm(x.data_ptr(), pr, pw, pb, y.data_ptr(), _address(summed), mean.data_ptr(), rstd.data_ptr(),
                            _address(packed), rows, hidden, eps, kind, DTYPES[pdtype], block, _code(code)), handle)
        return rc, LayerNorm(y, mean, rstd, summed, packed)

    rc, result = _run(device, stream, call)
    if rc:
        _check(rc, "taco_layernorm")
    return result


def layernorm_backward(dy: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       x: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                       packed: Optional[torch.Tensor] = None, dsummed: Optional[torch.Tensor] = None,
                       block: int = 128, code="e4m3", bias_grad: bool = True, stream=None,
                       bias_dtype: Optional[torch.dtype] = None) -> LayerNormGrads:
    """Gradients of layernorm from either (x, mean), x being what was
    normalised (`summed` where there was a residual), or the records `packed`.
    dsummed, the gradient that reaches `summed` from elsewhere, is added to dx.
    dweight is in weight's type, and None without a weight.  dbias is in that
    type too; the bias of a norm without a weight has its gradient in
    bias_dtype.  It is None with neither, and with bias_grad=False."""
    if bias_dtype is not None and bias_dtype not in DTYPES:
        raise TypeError(f"bias_dtype must be bfloat16, float16 or float32, got {bias_dtype}")
    if (x is None) == (packed is None) or (x is None) != (mean is None):
        raise ValueError("give either x with mean, or packed")
    kind, rows, hidden = _first(dy, "dy")
    device, shape, stats = dy.get_device(), dy.shape, dy.shape[:-1]
    if weight is None:
        pdtype = bias_dtype or torch.float32
    else:
        pdtype = _param_type(weight, "weight")
        if bias_dtype is not None and bias_dtype is not pdtype:
            raise TypeError(f"bias_dtype must be weight's type {pdtype}, got {bias_dtype}")
    bias_grad = bias_grad and (weight is not None or bias_dtype is not None)
    prstd = _tensor(rstd, "rstd", device, torch.float32, stats)
    px = _tensor(x, "x", device, dy.dtype, shape)
    pmean = _tensor(mean, "mean", device, torch.float32, stats)
    ppacked = 0 if packed is None else _packed(packed, rows, hidden, block, device)
    pw = _tensor(weight, "weight", device, pdtype, (hidden,))
    pds = _tensor(dsummed, "dsummed", device, dy.dtype, shape)
    lib = _library()

    def call(handle):
        dx = torch.empty_like(dy)
        dweight = dbias = ws = None
        nbytes = 0
        if weight is not None or bias_grad:
            dweight = torch.empty_like(weight) if weight is not None else None
            dbias = torch.empty(hidden, dtype=pdtype, device=dy.device) if bias_grad else None
            nbytes = _workspace_bytes("taco_layernorm_backward_workspace", rows, hidden)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
        rc = lib.taco_layernorm_backward(
            _pack_layernorm_backward(dy.data_ptr(), px, pmean, prstd, ppacked, pw, pds, dx.data_ptr(), _address(dweight),
                                     _address(dbias), _address(ws), nbytes, rows, hidden, kind, DTYPES[pdtype], block,
                                     _code(code)), handle)
        return rc, LayerNormGrads(dx, dweight, dbias)

    rc, result = _run(device, stream, call)
    if rc:
        _check(rc, "taco_layernorm_backward")
    return result


def _tanh_form(approximate: str) -> int:
    if approximate not in ("none", "tanh"):
        raise ValueError(f"approximate must be 'none' or 'tanh', got {approximate!r}")
    return int(approximate == "tanh")


def gelu(x: torch.Tensor, bias: Optional[torch.Tensor] = None, approximate: str = "none", checkpoint: bool = True,
         block: int = 128, code="e4m3", stream=None) -> Gelu:
    """GELU of u = x + bias (added in float32), and the 8-bit records of u."""
    tanh_form = _tanh_form(approximate)
    kind, rows, hidden = _first(x, "x")
    device = x.get_device()
    pdtype = _param_type(bias, "bias")
    pb = _tensor(bias, "bias", device, pdtype, (hidden,))
    nbytes = _record_bytes(rows, hidden, block) if checkpoint else 0

    def call(handle):
        y = torch.empty_like(x)
        packed = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if checkpoint else None
        rc = _library().taco_gelu(_pack_gelu(x.data_ptr(), pb, y.data_ptr(), _address(packed), rows, hidden, kind, DTYPES[pdtype],
                                             tanh_form, block, _code(code)), handle)
        return rc, Gelu(y, packed)

    rc, result = _run(device, stream, call)
    if rc:
        _check(rc, "taco_gelu")
    return result


def gelu_backward(dy: torch.Tensor, packed: torch.Tensor, approximate: str = "none",
                  bias_dtype: Optional[torch.dtype] = None, recompute: bool = False, block: int = 128, code="e4m3",
                  stream=None) -> GeluGrads:
    """Gradient of gelu from its records.  With bias_dtype the bias gradient
    (the sum of dx over rows) in that type; with recompute the activation y
    again, for the next layer's weight gradient."""
    tanh_form = _tanh_form(approximate)
    if bias_dtype is not None and bias_dtype not in DTYPES:
        raise TypeError(f"bias_dtype must be bfloat16, float16 or float32, got {bias_dtype}")
    kind, rows, hidden = _first(dy, "dy")
    device = dy.get_device()
    ppacked = _packed(packed, rows, hidden, block, device)
    lib = _library()

    def call(handle):
        dx = torch.empty_like(dy)
        y = torch.empty_like(dy) if recompute else None
        dbias = ws = None
        nbytes = 0
        if bias_dtype is not None:
            dbias = torch.empty(hidden, dtype=bias_dtype, device=dy.device)
            nbytes = _workspace_bytes("taco_gelu_backward_workspace", rows, hidden)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
        rc = lib.taco_gelu_backward(
            _pack_gelu_backward(dy.data_ptr(), ppacked, dx.data_ptr(), _address(y), _address(dbias), _address(ws), nbytes, rows,
                                hidden, kind, DTYPES[bias_dtype or torch.float32], tanh_form, block, _code(code)), handle)
        return rc, GeluGrads(dx, dbias, y)

    rc, result = _run(device, stream, call)
    if rc:
        _check(rc, "taco_gelu_backward")
    return result


def weight_grad(dy: torch.Tensor, packed: torch.Tensor, hidden: int, block: int = 128, code="e4m3",
                scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                dy_sum: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """dy^T X, the weight gradient [out features, hidden] of a linear layer
    whose input X [rows, hidden] was kept as records.  With scale and shift (a
    layer norm's weight and bias) X stands for X scale + shift; shift needs
    dy_sum, the float32 sum of dy over rows (the layer's bias gradient).  The
    result has `dtype` (float32 or bfloat16), or goes to `out`, to which
    accumulate=True adds it.  The checkpoints of layernorm and gelu enter the
    product as they are; records of compress(variant="ds_only"), whose scales
    are no powers of two, are rounded to bfloat16 for it (2^-9 of a value at
    most)."""
    kind, rows, features = _first(dy, "dy")
    if kind != 0:
        raise TypeError(f"dy must be torch.bfloat16, got {dy.dtype}")
    if (shift is None) != (dy_sum is None):
        raise ValueError("shift and dy_sum belong together")
    device = dy.get_device()
    ppacked = _packed(packed, rows, hidden, block, device)
    pdtype = _param_type(scale if scale is not None else shift, "scale")
    pscale = _tensor(scale, "scale", device, pdtype, (hidden,))
    pshift = _tensor(shift, "shift", device, pdtype, (hidden,))
    psum = _tensor(dy_sum, "dy_sum", device, torch.float32, (features,))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
    else:
        dtype = out.dtype
        _tensor(out, "out", device, dtype, (features, hidden))
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError(f"the gradient must be float32 or bfloat16, got {dtype}")
    lib = _library()

    def call(handle):
        dw = torch.empty((features, hidden), dtype=dtype, device=dy.device) if out is None else out
        nbytes = _workspace_bytes("taco_weight_grad_workspace", rows, features, hidden)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
        rc = lib.taco_weight_grad(
            _pack_weight_grad(dy.data_ptr(), ppacked, dw.data_ptr(), pscale, pshift, psum, _address(ws), nbytes, rows, features,
                              hidden, DTYPES[dtype], DTYPES[pdtype], int(accumulate), block, _code(code)), handle)
        return rc, dw

    rc, result = _run(device, stream, call)
    if rc:
        _check(rc, "taco_weight_grad")
    return result
