"""The longest sums of the gated layer's products: what they may take is bounded by
the kernels' waits, so longer ones are refused on the host.  A misplaced pointer,
which is looked at behind the sizes, shows that the others are let through."""
import ctypes

import pytest

from test_gated_refusals import A, ALIGN, CALLS, DEFAULTS, SHAPE, t  # noqa: F401

LONGEST = 1 << 24


@pytest.mark.parametrize("kind,change,status", [
    ("_GatedLinearArgs", dict(hidden=LONGEST, x=(1 << 40) + 8), ALIGN),
    ("_GatedLinearArgs", dict(hidden=LONGEST + 8, x=(1 << 40) + 8), SHAPE),
    ("_GatedLinearArgs", dict(hidden=LONGEST + 1), SHAPE),
    ("_GatedLinearArgs", dict(hidden=(1 << 31) - 257), SHAPE),
    ("_GatedLinearArgs", dict(hidden=230_000_000, rows=1, inner=32, block=32, packed=5 * A), SHAPE),
    ("_GatedLinearArgs", dict(hidden=LONGEST + 8, rows=0), SHAPE),
    ("_GatedLinearArgs", dict(inner=1 << 24, y=(1 << 40) + 8), ALIGN),
    ("_GatedLinearBackwardArgs", dict(inner=LONGEST // 2, dz=(1 << 40) + 8), ALIGN),
    ("_GatedLinearBackwardArgs", dict(inner=LONGEST // 2 + 128, dz=(1 << 40) + 8), SHAPE),
    ("_GatedLinearBackwardArgs", dict(inner=LONGEST // 2 + 128, weight=None, dx=None, dz=(1 << 40) + 8), ALIGN),
    ("_GatedLinearBackwardArgs", dict(hidden=LONGEST + 8, dz=(1 << 40) + 8), ALIGN),
])
def test_longest_sum(t, kind, change, status):  # noqa: F811
    args = getattr(t, kind)(**{**DEFAULTS[kind], **change})
    assert getattr(t._library(), CALLS[kind])(ctypes.byref(args), None) == status


def test_workspace_queries(t):  # noqa: F811
    lib = t._library()
    assert lib.taco_gated_linear_workspace(16, 64, LONGEST) == 0
    assert lib.taco_gated_linear_workspace(16, 64, LONGEST - 1) > 0
    assert lib.taco_gated_linear_workspace(16, 64, LONGEST + 1) == -1
    assert lib.taco_gated_linear_backward_workspace(16, LONGEST // 2, 64) > 0
    assert lib.taco_gated_linear_backward_workspace(16, LONGEST // 2 + 1, 64) == -1
    assert lib.taco_gated_linear_backward_workspace(16, LONGEST // 2 + 1, 0) > 0
    assert lib.taco_gated_linear_backward_workspace(16, 64, LONGEST + 1) > 0
