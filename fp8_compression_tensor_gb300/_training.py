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
Argument marshalling only, like _binding.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional

import torch

from ._binding import CODES, _check, _check_cuda_tensor, _stream_handle, compressed_bytes, load_library

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


_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = load_library()
        for name, args in (("taco_layernorm", _LayerNormArgs), ("taco_layernorm_backward", _LayerNormBackwardArgs),
                           ("taco_gelu", _GeluArgs), ("taco_gelu_backward", _GeluBackwardArgs),
                           ("taco_weight_grad", _WeightGradArgs)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [ctypes.POINTER(args), _ptr], _i32
        for name in ("taco_layernorm_backward_workspace", "taco_gelu_backward_workspace"):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [_i64, _i64], _i64
        lib.taco_weight_grad_workspace.argtypes, lib.taco_weight_grad_workspace.restype = [_i64, _i64, _i64], _i64
        _lib = lib
    return _lib


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


def _tensor(t, name: str, like: torch.Tensor, dtype=None, shape=None) -> int:
    """Checks one tensor argument (None passes) and returns its address."""
    if t is None:
        return None
    _check_cuda_tensor(t, t.dtype if dtype is None and isinstance(t, torch.Tensor) else dtype, name)
    if t.dtype not in DTYPES and t.dtype != torch.uint8:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    return t.data_ptr()


def _rows_hidden(x: torch.Tensor):
    if x.dim() == 0:
        raise ValueError("tensor must have at least one dimension")
    return math.prod(x.shape[:-1]), x.shape[-1]


def _packed(packed: torch.Tensor, rows: int, hidden: int, block: int, like: torch.Tensor) -> int:
    address = _tensor(packed, "packed", like, torch.uint8)
    nbytes = compressed_bytes(rows, hidden, block)
    if packed.numel() != nbytes:
        raise ValueError(f"packed must have {nbytes} bytes, has {packed.numel()}")
    return address


class _On(contextlib.ExitStack):
    """The device and the stream that a call runs on; tensors allocated inside
    belong to that stream, so one that is freed while the call still runs (a
    workspace) is reused behind it only."""

    def __init__(self, device: torch.device, stream):
        super().__init__()
        if device.index != torch.cuda.current_device():
            self.enter_context(torch.cuda.device(device))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.enter_context(torch.cuda.stream(stream))
        self.handle = _stream_handle(device, stream)


def layernorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              eps: float = 1e-5, residual: Optional[torch.Tensor] = None, checkpoint: bool = False, block: int = 128,
              code="e4m3", stream=None) -> LayerNorm:
    """Layer norm over the last dimension of x (bf16, f16 or f32), or of
    x + residual (rounded to x's type and returned as `summed`).  weight and
    bias share one type.  mean and rstd are float32, one per row.  With
    checkpoint, `packed` holds the normalised rows (before weight and bias) as
    8-bit records."""
    px = _tensor(x, "x", x)
    rows, hidden = _rows_hidden(x)
    pr = _tensor(residual, "residual", x, x.dtype, x.shape)
    param = weight if weight is not None else bias
    pdtype = param.dtype if param is not None else torch.float32
    pw = _tensor(weight, "weight", x, pdtype, (hidden,))
    pb = _tensor(bias, "bias", x, pdtype, (hidden,))
    nbytes = compressed_bytes(rows, hidden, block) if checkpoint else 0
    with _On(x.device, stream) as on:
        y = torch.empty_like(x)
        summed = torch.empty_like(x) if residual is not None else None
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        packed = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if checkpoint else None
        args = _LayerNormArgs(px, pr, pw, pb, y.data_ptr(), None if summed is None else summed.data_ptr(),
                              mean.data_ptr(), rstd.data_ptr(), packed.data_ptr() if checkpoint else None, rows, hidden,
                              eps, DTYPES[x.dtype], DTYPES[pdtype], block, _code(code))
        rc = _library().taco_layernorm(args, on.handle)
    _check(rc, "taco_layernorm")
    return LayerNorm(y, mean, rstd, summed, packed)


def layernorm_backward(dy: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       x: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                       packed: Optional[torch.Tensor] = None, dsummed: Optional[torch.Tensor] = None,
                       block: int = 128, code="e4m3", bias_grad: bool = True, stream=None) -> LayerNormGrads:
    """Gradients of layernorm from either (x, mean), x being what was
    normalised (`summed` where there was a residual), or the records `packed`.
    dsummed, the gradient that reaches `summed` from elsewhere, is added to dx.
    dweight and dbias (in weight's type) are None without a weight; dbias also
    with bias_grad=False."""
    if (x is None) == (packed is None) or (x is None) != (mean is None):
        raise ValueError("give either x with mean, or packed")
    pdy = _tensor(dy, "dy", dy)
    rows, hidden = _rows_hidden(dy)
    prstd = _tensor(rstd, "rstd", dy, torch.float32, dy.shape[:-1])
    px = _tensor(x, "x", dy, dy.dtype, dy.shape)
    pmean = _tensor(mean, "mean", dy, torch.float32, dy.shape[:-1])
    ppacked = None if packed is None else _packed(packed, rows, hidden, block, dy)
    pw = _tensor(weight, "weight", dy, None, (hidden,))
    pds = _tensor(dsummed, "dsummed", dy, dy.dtype, dy.shape)
    lib = _library()
    with _On(dy.device, stream) as on:
        dx = torch.empty_like(dy)
        dweight = torch.empty_like(weight) if weight is not None else None
        dbias = torch.empty_like(weight) if weight is not None and bias_grad else None
        nbytes = lib.taco_layernorm_backward_workspace(rows, hidden) if weight is not None else 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
        args = _LayerNormBackwardArgs(
            pdy, px, pmean, prstd, ppacked, pw, pds, dx.data_ptr(), None if dweight is None else dweight.data_ptr(),
            None if dbias is None else dbias.data_ptr(), None if ws is None else ws.data_ptr(), nbytes, rows, hidden,
            DTYPES[dy.dtype], DTYPES[torch.float32 if weight is None else weight.dtype], block, _code(code))
        rc = lib.taco_layernorm_backward(args, on.handle)
    _check(rc, "taco_layernorm_backward")
    return LayerNormGrads(dx, dweight, dbias)


def _tanh_form(approximate: str) -> int:
    if approximate not in ("none", "tanh"):
        raise ValueError(f"approximate must be 'none' or 'tanh', got {approximate!r}")
    return int(approximate == "tanh")


def gelu(x: torch.Tensor, bias: Optional[torch.Tensor] = None, approximate: str = "none", checkpoint: bool = True,
         block: int = 128, code="e4m3", stream=None) -> Gelu:
    """GELU of u = x + bias (added in float32), and the 8-bit records of u."""
    tanh_form = _tanh_form(approximate)
    px = _tensor(x, "x", x)
    rows, hidden = _rows_hidden(x)
    pb = _tensor(bias, "bias", x, None, (hidden,))
    nbytes = compressed_bytes(rows, hidden, block) if checkpoint else 0
    with _On(x.device, stream) as on:
        y = torch.empty_like(x)
        packed = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if checkpoint else None
        args = _GeluArgs(px, pb, y.data_ptr(), packed.data_ptr() if checkpoint else None, rows, hidden, DTYPES[x.dtype],
                         DTYPES[torch.float32 if bias is None else bias.dtype], tanh_form, block, _code(code))
        rc = _library().taco_gelu(args, on.handle)
    _check(rc, "taco_gelu")
    return Gelu(y, packed)


def gelu_backward(dy: torch.Tensor, packed: torch.Tensor, approximate: str = "none",
                  bias_dtype: Optional[torch.dtype] = None, recompute: bool = False, block: int = 128, code="e4m3",
                  stream=None) -> GeluGrads:
    """Gradient of gelu from its records.  With bias_dtype the bias gradient
    (the sum of dx over rows) in that type; with recompute the activation y
    again, for the next layer's weight gradient."""
    tanh_form = _tanh_form(approximate)
    if bias_dtype is not None and bias_dtype not in DTYPES:
        raise TypeError(f"bias_dtype must be bfloat16, float16 or float32, got {bias_dtype}")
    pdy = _tensor(dy, "dy", dy)
    rows, hidden = _rows_hidden(dy)
    ppacked = _packed(packed, rows, hidden, block, dy)
    lib = _library()
    with _On(dy.device, stream) as on:
        dx = torch.empty_like(dy)
        y = torch.empty_like(dy) if recompute else None
        dbias = torch.empty(hidden, dtype=bias_dtype, device=dy.device) if bias_dtype is not None else None
        nbytes = lib.taco_gelu_backward_workspace(rows, hidden) if bias_dtype is not None else 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
        args = _GeluBackwardArgs(
            pdy, ppacked, dx.data_ptr(), None if y is None else y.data_ptr(), None if dbias is None else dbias.data_ptr(),
            None if ws is None else ws.data_ptr(), nbytes, rows, hidden, DTYPES[dy.dtype],
            DTYPES[torch.float32 if bias_dtype is None else bias_dtype], tanh_form, block, _code(code))
        rc = lib.taco_gelu_backward(args, on.handle)
    _check(rc, "taco_gelu_backward")
    return GeluGrads(dx, dbias, y)


def weight_grad(dy: torch.Tensor, packed: torch.Tensor, hidden: int, block: int = 128, code="e4m3",
                scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                dy_sum: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """dy^T X, the weight gradient [out features, hidden] of a linear layer
    whose input X [rows, hidden] was kept as records.  With scale and shift (a
    layer norm's weight and bias) X stands for X scale + shift; shift needs
    dy_sum, the float32 sum of dy over rows (the layer's bias gradient).  The
    result has `dtype` (float32 or bfloat16), or goes to `out`, to which
    accumulate=True adds it."""
    pdy = _tensor(dy, "dy", dy, torch.bfloat16)
    rows, features = _rows_hidden(dy)
    ppacked = _packed(packed, rows, hidden, block, dy)
    if (shift is None) != (dy_sum is None):
        raise ValueError("shift and dy_sum belong together")
    param = scale if scale is not None else shift
    pdtype = param.dtype if param is not None else torch.float32
    pscale = _tensor(scale, "scale", dy, pdtype, (hidden,))
    pshift = _tensor(shift, "shift", dy, pdtype, (hidden,))
    psum = _tensor(dy_sum, "dy_sum", dy, torch.float32, (features,))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
    else:
        dtype = out.dtype
        _tensor(out, "out", dy, dtype, (features, hidden))
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"the gradient must be float32 or bfloat16, got {dtype}")
    lib = _library()
    with _On(dy.device, stream) as on:
        if out is None:
            out = torch.empty((features, hidden), dtype=dtype, device=dy.device)
        nbytes = lib.taco_weight_grad_workspace(rows, features, hidden)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device) if nbytes > 0 else None
        args = _WeightGradArgs(pdy, ppacked, out.data_ptr(), pscale, pshift, psum, None if ws is None else ws.data_ptr(),
                               max(nbytes, 0), rows, features, hidden, DTYPES[dtype], DTYPES[pdtype], int(accumulate), block,
                               _code(code))
        rc = lib.taco_weight_grad(args, on.handle)
    _check(rc, "taco_weight_grad")
    return out
