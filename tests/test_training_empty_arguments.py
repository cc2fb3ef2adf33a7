"""The training calls of the C ABI on empty tensors, whose pointers may be null:
sizes are looked at before the pointers that belong together (CPU)."""
import ctypes

import pytest

from test_training_refusals import A, BLOCK, CALLS, DEFAULTS, OK, OPTIONS, t  # noqa: F401


@pytest.mark.parametrize("kind,change,status", [
    ("_LayerNormBackwardArgs", dict(hidden=0, x=None, dy=None, dx=None), OK),
    ("_LayerNormBackwardArgs", dict(hidden=0, x=None, mean=None, packed=None, dy=None, dx=None), OK),
    ("_LayerNormBackwardArgs", dict(hidden=0, x=None, mean=None, block=7), BLOCK),
    ("_LayerNormBackwardArgs", dict(rows=0, x=None, mean=None, dy=None), OK),
    ("_LayerNormBackwardArgs", dict(x=None), OPTIONS),
    ("_LayerNormBackwardArgs", dict(mean=None), OPTIONS),
    ("_WeightGradArgs", dict(out=0, shift=5 * A, dy_sum=None, dy=None), OK),
    ("_WeightGradArgs", dict(hidden=0, shift=None, dy_sum=5 * A, packed=None), OK),
    ("_WeightGradArgs", dict(rows=0, out=0, shift=5 * A, dy_sum=None), OK),
    ("_WeightGradArgs", dict(rows=0, shift=5 * A, dy_sum=None), OPTIONS),
    ("_WeightGradArgs", dict(shift=5 * A), OPTIONS),
    ("_WeightGradArgs", dict(dy_sum=5 * A), OPTIONS),
])
def test_sizes_before_pairs(t, kind, change, status):  # noqa: F811
    args = getattr(t, kind)(**{**DEFAULTS[kind], **change})
    assert getattr(t._library(), CALLS[kind])(ctypes.byref(args), None) == status
