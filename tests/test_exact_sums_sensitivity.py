"""The inputs of exact_sums.py show a mistake in a long sum: one planted in the
expected values, a stage of 64 terms left out or taken twice of 32768, changes most outputs."""
import pytest
import torch

import exact_sums as ex


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float16))
@pytest.mark.parametrize("columns", (slice(0, 64), slice(32704, 32768), slice(8192, 8256)))
def test_layer(dtype, columns):
    x, w, bias = ex.layer(20, 32768, 16)
    y = ex.layer_values(x, w, bias)[1].to(dtype)
    for factor in (0, 2):
        planted = x.clone()
        planted[:, columns] *= factor
        # what the sum of the up projection loses is several hundredths of it, as a rule
        assert (ex.layer_values(planted, w, bias)[1].to(dtype) != y).float().mean() > 0.8


@pytest.mark.parametrize("rows_of_w", (slice(0, 64), slice(32704, 32768)))
def test_gradient(rows_of_w):
    dy, up, w = ex.gradient(20, 24, 16384)
    dz, dx, _ = ex.gradient_values(dy, up, w)
    planted = w.clone()
    planted[rows_of_w] = 0
    wrong = ex.gradient_values(dy, up, planted)[1]
    # a gate's stage adds 5 to sums of 2700, an up projection's 170
    assert (wrong.to(torch.bfloat16) != dx.to(torch.bfloat16)).float().mean() > 0.2
