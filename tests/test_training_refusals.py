"""The training calls of the C ABI check their arguments on the host, before
any device call; their workspace queries need no device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def t():
    from fp8_compression_tensor_gb300 import build
    build.build()
    from fp8_compression_tensor_gb300 import _training
    _training._library()
    return _training


OK, NULL, SHAPE, BLOCK, ALIGN, OVERLAP, OPTIONS = 0, 1, 2, 3, 4, 6, 9
A = 1 << 20   # addresses a MiB apart that no check reads
DEFAULTS = {
    "_LayerNormArgs": dict(x=A, y=2 * A, mean=3 * A, rstd=4 * A, rows=4, hidden=256, eps=1e-5, dtype=0, param_dtype=2,
                           block=128, code=0),
    "_LayerNormBackwardArgs": dict(dy=A, x=2 * A, mean=3 * A, rstd=4 * A, dx=5 * A, rows=4, hidden=256, dtype=0,
                                   param_dtype=2, block=128, code=0),
    "_GeluArgs": dict(x=A, y=2 * A, rows=4, hidden=256, dtype=0, param_dtype=2, tanh_form=0, block=128, code=0),
    "_GeluBackwardArgs": dict(dy=A, packed=2 * A, dx=3 * A, rows=4, hidden=256, dtype=0, param_dtype=2, tanh_form=0,
                              block=128, code=0),
    "_WeightGradArgs": dict(dy=A, packed=2 * A, dweight=3 * A, rows=4, out=64, hidden=256, dtype=2, param_dtype=2,
                            accumulate=0, block=128, code=0, workspace=8 * A, workspace_bytes=1 << 40),
}
CALLS = {"_LayerNormArgs": "taco_layernorm", "_LayerNormBackwardArgs": "taco_layernorm_backward",
         "_GeluArgs": "taco_gelu", "_GeluBackwardArgs": "taco_gelu_backward", "_WeightGradArgs": "taco_weight_grad"}


@pytest.mark.parametrize("kind", sorted(CALLS))
def test_null_arguments(t, kind):
    assert getattr(t._library(), CALLS[kind])(None, None) == OPTIONS


@pytest.mark.parametrize("kind,change,status", [
    ("_LayerNormArgs", dict(dtype=3), OPTIONS),
    ("_LayerNormArgs", dict(param_dtype=-1), OPTIONS),
    ("_LayerNormArgs", dict(eps=-1.0), OPTIONS),
    ("_LayerNormArgs", dict(eps=float("nan")), OPTIONS),
    ("_LayerNormArgs", dict(residual=5 * A), OPTIONS),
    ("_LayerNormArgs", dict(summed=5 * A), OPTIONS),
    ("_LayerNormArgs", dict(rows=-1), SHAPE),
    ("_LayerNormArgs", dict(hidden=-1), SHAPE),
    ("_LayerNormArgs", dict(rows=1 << 40, hidden=1 << 40), SHAPE),
    ("_LayerNormArgs", dict(packed=5 * A, code=3), OPTIONS),
    ("_LayerNormArgs", dict(packed=5 * A, block=96), BLOCK),
    ("_LayerNormArgs", dict(packed=5 * A, block=512), SHAPE),
    ("_LayerNormArgs", dict(x=None), NULL),
    ("_LayerNormArgs", dict(rstd=None), NULL),
    ("_LayerNormArgs", dict(x=A + 8), ALIGN),
    ("_LayerNormArgs", dict(weight=5 * A + 4), ALIGN),
    ("_LayerNormArgs", dict(y=A), OVERLAP),
    ("_LayerNormArgs", dict(packed=2 * A + 1024), OVERLAP),
    ("_LayerNormArgs", dict(mean=4 * A), OVERLAP),
    ("_LayerNormArgs", dict(rows=0, x=None), OK),
    ("_LayerNormArgs", dict(hidden=0, x=None), OK),
    ("_LayerNormBackwardArgs", dict(mean=None), OPTIONS),
    ("_LayerNormBackwardArgs", dict(x=None), OPTIONS),
    ("_LayerNormBackwardArgs", dict(packed=6 * A), OPTIONS),
    ("_LayerNormBackwardArgs", dict(x=None, mean=None), NULL),
    ("_LayerNormBackwardArgs", dict(x=None, mean=None, packed=6 * A, block=7), BLOCK),
    ("_LayerNormBackwardArgs", dict(x=None, mean=None, packed=6 * A, hidden=100), SHAPE),
    ("_LayerNormBackwardArgs", dict(dweight=7 * A), NULL),
    ("_LayerNormBackwardArgs", dict(dweight=7 * A, workspace=8 * A, workspace_bytes=16), SHAPE),
    ("_LayerNormBackwardArgs", dict(dx=A), OVERLAP),
    ("_LayerNormBackwardArgs", dict(dweight=7 * A, workspace=7 * A, workspace_bytes=1 << 20), OVERLAP),
    ("_LayerNormBackwardArgs", dict(dx=5 * A + 2), ALIGN),
    ("_LayerNormBackwardArgs", dict(rows=0, dy=None), OK),
    ("_GeluArgs", dict(tanh_form=2), OPTIONS),
    ("_GeluArgs", dict(dtype=-1), OPTIONS),
    ("_GeluArgs", dict(packed=3 * A, block=33), BLOCK),
    ("_GeluArgs", dict(packed=3 * A, hidden=130), SHAPE),
    ("_GeluArgs", dict(packed=3 * A, hidden=1 << 31), SHAPE),
    ("_GeluArgs", dict(hidden=1 << 31, y=None), NULL),
    ("_GeluArgs", dict(y=None), NULL),
    ("_GeluArgs", dict(bias=3 * A + 2), ALIGN),
    ("_GeluArgs", dict(packed=A + 512), OVERLAP),
    ("_GeluBackwardArgs", dict(code=-1), OPTIONS),
    ("_GeluBackwardArgs", dict(hidden=130), SHAPE),
    ("_GeluBackwardArgs", dict(packed=None), NULL),
    ("_GeluBackwardArgs", dict(dbias=4 * A), NULL),
    ("_GeluBackwardArgs", dict(dbias=4 * A, workspace=5 * A, workspace_bytes=100), SHAPE),
    ("_GeluBackwardArgs", dict(y=3 * A), OVERLAP),
    ("_WeightGradArgs", dict(dtype=1), OPTIONS),
    ("_WeightGradArgs", dict(accumulate=2), OPTIONS),
    ("_WeightGradArgs", dict(shift=5 * A), OPTIONS),
    ("_WeightGradArgs", dict(dy_sum=5 * A), OPTIONS),
    ("_WeightGradArgs", dict(out=-1), SHAPE),
    ("_WeightGradArgs", dict(rows=1 << 32, out=8, hidden=128), SHAPE),
    ("_WeightGradArgs", dict(block=48), BLOCK),
    ("_WeightGradArgs", dict(dy=None), NULL),
    ("_WeightGradArgs", dict(scale=5 * A + 8), ALIGN),
    ("_WeightGradArgs", dict(dweight=A), OVERLAP),
    ("_WeightGradArgs", dict(out=0, dy=None, packed=None), OK),
    ("_WeightGradArgs", dict(hidden=0, dy=None, packed=None), OK),
])
def test_argument_checks(t, kind, change, status):
    args = getattr(t, kind)(**{**DEFAULTS[kind], **change})
    assert getattr(t._library(), CALLS[kind])(ctypes.byref(args), None) == status


def test_workspace_queries(t):
    lib = t._library()
    assert lib.taco_layernorm_backward_workspace(0, 4096) == 0
    assert 0 < lib.taco_layernorm_backward_workspace(1, 1) <= 1 << 16
    assert lib.taco_layernorm_backward_workspace(-1, 4) == -1
    assert lib.taco_layernorm_backward_workspace(1 << 40, 1 << 40) == -1
    assert lib.taco_gelu_backward_workspace(8192, 16384) >= 4 * 16384
    assert lib.taco_gelu_backward_workspace(4, -1) == -1
    assert lib.taco_weight_grad_workspace(16, -1, 128) == -1
    assert lib.taco_weight_grad_workspace(16, 64, 128) >= 0


def test_binding_refuses_cpu_tensors():
    import torch
    import fp8_compression_tensor_gb300 as taco
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        taco.layernorm(x)
    with pytest.raises(TypeError):
        taco.gelu(x)
    with pytest.raises(TypeError):
        taco.weight_grad(x, x, 128)
