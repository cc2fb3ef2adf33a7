"""The RMS norm and the gated linear layer of the C ABI check their arguments on
the host, before any device call; their workspace queries need no device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def t():
    from fp8_compression_tensor_gb300 import build
    build.build()
    from fp8_compression_tensor_gb300 import _gated
    _gated._library()
    return _gated


OK, NULL, SHAPE, BLOCK, ALIGN, OVERLAP, OPTIONS = 0, 1, 2, 3, 4, 6, 9
A = 1 << 20   # addresses a MiB apart that no check reads
WORK = dict(workspace=64 * A, workspace_bytes=1 << 40)
DEFAULTS = {
    "_RmsNormArgs": dict(x=A, y=2 * A, rstd=3 * A, rows=4, hidden=256, eps=1e-6, dtype=0, param_dtype=2, block=128, code=0),
    "_RmsNormBackwardArgs": dict(dy=A, x=2 * A, rstd=3 * A, dx=4 * A, rows=4, hidden=256, dtype=0, param_dtype=2, block=128,
                                 code=0),
    "_GatedLinearArgs": dict(x=A, weight=2 * A, y=3 * A, rows=4, inner=256, hidden=64, dtype=0, param_dtype=2, activation=0,
                             block=128, code=0, **WORK),
    "_GatedLinearBackwardArgs": dict(dy=A, packed=2 * A, weight=3 * A, dz=4 * A, dx=5 * A, rows=4, inner=256, hidden=64,
                                     dtype=0, param_dtype=2, activation=0, block=128, code=0, **WORK),
}
CALLS = {"_RmsNormArgs": "taco_rmsnorm", "_RmsNormBackwardArgs": "taco_rmsnorm_backward",
         "_GatedLinearArgs": "taco_gated_linear", "_GatedLinearBackwardArgs": "taco_gated_linear_backward"}


@pytest.mark.parametrize("kind", sorted(CALLS))
def test_null_arguments(t, kind):
    assert getattr(t._library(), CALLS[kind])(None, None) == OPTIONS


@pytest.mark.parametrize("kind,change,status", [
    ("_RmsNormArgs", dict(dtype=3), OPTIONS),
    ("_RmsNormArgs", dict(param_dtype=-1), OPTIONS),
    ("_RmsNormArgs", dict(eps=-1.0), OPTIONS),
    ("_RmsNormArgs", dict(eps=float("nan")), OPTIONS),
    ("_RmsNormArgs", dict(residual=5 * A), OPTIONS),
    ("_RmsNormArgs", dict(summed=5 * A), OPTIONS),
    ("_RmsNormArgs", dict(packed_y=5 * A), OPTIONS),
    ("_RmsNormArgs", dict(rows=-1), SHAPE),
    ("_RmsNormArgs", dict(hidden=-1), SHAPE),
    ("_RmsNormArgs", dict(rows=1 << 40, hidden=1 << 40), SHAPE),
    ("_RmsNormArgs", dict(packed=5 * A, code=3), OPTIONS),
    ("_RmsNormArgs", dict(packed=5 * A, block=96), BLOCK),
    ("_RmsNormArgs", dict(packed=5 * A, block=512), SHAPE),
    ("_RmsNormArgs", dict(y=None, packed_y=5 * A, hidden=100), SHAPE),
    ("_RmsNormArgs", dict(y=None), NULL),
    ("_RmsNormArgs", dict(x=None), NULL),
    ("_RmsNormArgs", dict(rstd=None), NULL),
    ("_RmsNormArgs", dict(x=A + 8), ALIGN),
    ("_RmsNormArgs", dict(weight=5 * A + 4), ALIGN),
    ("_RmsNormArgs", dict(y=A), OVERLAP),
    ("_RmsNormArgs", dict(packed=2 * A + 1024), OVERLAP),
    ("_RmsNormArgs", dict(y=None, packed_y=5 * A, packed=5 * A), OVERLAP),
    ("_RmsNormArgs", dict(residual=5 * A, summed=A), OVERLAP),
    ("_RmsNormArgs", dict(rows=0, x=None), OK),
    ("_RmsNormArgs", dict(hidden=0, x=None), OK),
    ("_RmsNormBackwardArgs", dict(packed=6 * A), OPTIONS),
    ("_RmsNormBackwardArgs", dict(x=None), NULL),
    ("_RmsNormBackwardArgs", dict(x=None, packed=6 * A, block=7), BLOCK),
    ("_RmsNormBackwardArgs", dict(x=None, packed=6 * A, hidden=100), SHAPE),
    ("_RmsNormBackwardArgs", dict(dweight=7 * A), NULL),
    ("_RmsNormBackwardArgs", dict(dweight=7 * A, workspace=8 * A, workspace_bytes=16), SHAPE),
    ("_RmsNormBackwardArgs", dict(dx=A), OVERLAP),
    ("_RmsNormBackwardArgs", dict(dweight=7 * A, workspace=7 * A, workspace_bytes=1 << 20), OVERLAP),
    ("_RmsNormBackwardArgs", dict(dx=4 * A + 2), ALIGN),
    ("_RmsNormBackwardArgs", dict(rows=0, dy=None), OK),
    ("_RmsNormBackwardArgs", dict(hidden=0, dy=None, x=None), OK),
    ("_GatedLinearArgs", dict(dtype=2), OPTIONS),
    ("_GatedLinearArgs", dict(dtype=-1), OPTIONS),
    ("_GatedLinearArgs", dict(param_dtype=3), OPTIONS),
    ("_GatedLinearArgs", dict(activation=3), OPTIONS),
    ("_GatedLinearArgs", dict(activation=-1), OPTIONS),
    ("_GatedLinearArgs", dict(rows=-1), SHAPE),
    ("_GatedLinearArgs", dict(hidden=0), SHAPE),
    ("_GatedLinearArgs", dict(inner=1 << 40), SHAPE),
    ("_GatedLinearArgs", dict(rows=1 << 31), SHAPE),
    ("_GatedLinearArgs", dict(packed=5 * A, code=3), OPTIONS),
    ("_GatedLinearArgs", dict(packed=5 * A, block=256), BLOCK),
    ("_GatedLinearArgs", dict(packed=5 * A, block=512), BLOCK),
    ("_GatedLinearArgs", dict(packed=5 * A, block=33), BLOCK),
    ("_GatedLinearArgs", dict(packed=5 * A, inner=192), SHAPE),
    ("_GatedLinearArgs", dict(x=None), NULL),
    ("_GatedLinearArgs", dict(weight=None), NULL),
    ("_GatedLinearArgs", dict(y=None), NULL),
    ("_GatedLinearArgs", dict(hidden=63, workspace=None), NULL),
    ("_GatedLinearArgs", dict(hidden=63, workspace_bytes=16), SHAPE),
    ("_GatedLinearArgs", dict(hidden=63, workspace=64 * A + 8), ALIGN),
    ("_GatedLinearArgs", dict(weight=2 * A + 8), ALIGN),
    ("_GatedLinearArgs", dict(bias=5 * A + 2), ALIGN),
    ("_GatedLinearArgs", dict(y=A), OVERLAP),
    ("_GatedLinearArgs", dict(packed=2 * A), OVERLAP),
    ("_GatedLinearArgs", dict(rows=0, x=None, y=None), OK),
    ("_GatedLinearArgs", dict(inner=0, weight=None, y=None), OK),
    ("_GatedLinearBackwardArgs", dict(dtype=2), OPTIONS),
    ("_GatedLinearBackwardArgs", dict(activation=7), OPTIONS),
    ("_GatedLinearBackwardArgs", dict(code=-1), OPTIONS),
    ("_GatedLinearBackwardArgs", dict(block=256), BLOCK),
    ("_GatedLinearBackwardArgs", dict(inner=192), SHAPE),
    ("_GatedLinearBackwardArgs", dict(inner=0), SHAPE),
    ("_GatedLinearBackwardArgs", dict(hidden=0), SHAPE),
    ("_GatedLinearBackwardArgs", dict(weight=None), OPTIONS),
    ("_GatedLinearBackwardArgs", dict(dx=None), OPTIONS),
    ("_GatedLinearBackwardArgs", dict(dy=None), NULL),
    ("_GatedLinearBackwardArgs", dict(packed=None), NULL),
    ("_GatedLinearBackwardArgs", dict(dz=None), NULL),
    ("_GatedLinearBackwardArgs", dict(dbias=6 * A, workspace=None), NULL),
    ("_GatedLinearBackwardArgs", dict(dbias=6 * A, workspace_bytes=100), SHAPE),
    ("_GatedLinearBackwardArgs", dict(dz=A), OVERLAP),
    ("_GatedLinearBackwardArgs", dict(dx=4 * A), OVERLAP),
    ("_GatedLinearBackwardArgs", dict(y=4 * A + 16), OVERLAP),
    ("_GatedLinearBackwardArgs", dict(dbias=6 * A, workspace=6 * A), OVERLAP),
    ("_GatedLinearBackwardArgs", dict(dz=4 * A + 8), ALIGN),
    ("_GatedLinearBackwardArgs", dict(rows=0, dy=None, packed=None), OK),
])
def test_argument_checks(t, kind, change, status):
    args = getattr(t, kind)(**{**DEFAULTS[kind], **change})
    assert getattr(t._library(), CALLS[kind])(ctypes.byref(args), None) == status


def test_workspace_queries(t):
    lib = t._library()
    assert lib.taco_rmsnorm_backward_workspace(0, 4096) == 0
    assert 0 < lib.taco_rmsnorm_backward_workspace(1, 1) <= 1 << 16
    assert lib.taco_rmsnorm_backward_workspace(-1, 4) == -1
    assert lib.taco_rmsnorm_backward_workspace(1 << 40, 1 << 40) == -1
    for query in (lib.taco_gated_linear_workspace, lib.taco_gated_linear_backward_workspace):
        assert query(16, -1, 128) == -1
        assert query(1 << 31, 8, 8) == -1
        assert query(16, 1 << 40, 1 << 40) == -1
        assert query(16, 64, 128) >= 0
    assert lib.taco_gated_linear_backward_workspace(8192, 16384, 0) >= 8 * 16384


def test_binding_refuses_bad_tensors():
    import torch
    import fp8_compression_tensor_gb300 as taco
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for call in (lambda: taco.rmsnorm(x), lambda: taco.rmsnorm_backward(x, x, x=x), lambda: taco.gated_linear(x, x),
                 lambda: taco.gated_linear_backward(x, x), lambda: taco.gated_linear_backward(x, x, bias_dtype=torch.int8)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        taco.gated_linear(x, x, activation="relu")
    with pytest.raises(ValueError):
        taco.rmsnorm_backward(x, x)
    with pytest.raises(ValueError):
        taco.rmsnorm_backward(x, x, x=x, packed=x)
