"""The way from the gated layer's gradient to its weight's: dz as it is written and
the records of the layer's input, with sums that are exact in binary32."""
import pytest
import torch

import exact_sums as ex
import training_reference as ref
from test_gpu_gated import BF16, F16, F32, taco  # noqa: F401

pytestmark = pytest.mark.gpu


def made(taco, rows, hidden, inner, dtype):
    dy, up, _ = ex.gradient(rows, 8, inner, device="cuda")
    z = torch.cat([torch.full_like(up, 32), up], 1).float()
    x = ex.signs(7, rows, hidden, density=2 / 3, device="cuda").float()
    g = taco.gated_linear_backward(dy.to(dtype), ref.make_records(z.cpu(), 128, "e4m3").cuda())
    return g.dz, x, ref.make_records(x.cpu(), 128, "e4m3").cuda()


@pytest.mark.parametrize("rows,hidden,inner", [(1, 128, 128), (300, 512, 384), (2049, 640, 128), (40, 128, 2560)])
def test_weight_gradient(taco, rows, hidden, inner):  # noqa: F811
    dz, x, packed = made(taco, rows, hidden, inner, BF16)
    want = dz.float().t() @ x          # whole numbers, of 32 times the rows at most
    assert torch.equal(taco.weight_grad(dz, packed, hidden), want)
    assert torch.equal(taco.weight_grad(dz, packed, hidden, scale=torch.full((hidden,), 0.5, device="cuda"), dtype=BF16),
                       (want / 2).to(BF16))


def test_weight_gradient_takes_bf16_alone(taco):  # noqa: F811
    dz, _, packed = made(taco, 8, 128, 128, F16)
    assert dz.dtype == F16
    with pytest.raises(TypeError, match="bfloat16"):
        taco.weight_grad(dz, packed, 128)
