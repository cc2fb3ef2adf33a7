"""GELU's vector kernel beyond one pass of its grid, where the bias column is
kept up by steps modulo the width, and without records at the widths, types and
forms that test_gpu_training leaves out.  64-bit references on the GPU, the
suite's bounds."""
import math

import numpy as np
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def check_value(y, u, tanh):
    u = u.double()
    want = (u * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)) if tanh
            else u * 0.5 * torch.erfc(-u / math.sqrt(2)))
    off = 8 * ref.U32 * u.abs()                           # training_reference.gelu_bound
    bound = off + ref.UNIT[y.dtype] * (want.abs() + off) + ref.TINY[y.dtype]
    assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("tanh", (False, True))
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("rows,hidden", [(2100, 5472), (131101, 88)])
def test_more_than_a_pass_of_the_grid(taco, tanh, dtype, pdtype, rows, hidden):
    """About 11.5 million elements; the widths divide neither the grid's step nor a warp's."""
    x, b = (2 * normal(1, rows, hidden)).to(dtype), normal(2, hidden).to(pdtype)
    u = x.float() + b.float()
    approximate = "tanh" if tanh else "none"
    check_value(taco.gelu(x, b, approximate=approximate, checkpoint=False).y, u, tanh)
    if hidden % 32 == 0:
        got = taco.gelu(x, b, approximate=approximate, block=32)
        check_value(got.y, u, tanh)
        val, s = ref.encode(ref.f64(u), 32, "e4m3")
        assert np.array_equal(ref.split(got.packed, 32)[2], s)
        assert np.array_equal(ref.decode(got.packed, rows, hidden, 32, "e4m3"), val)


@pytest.mark.parametrize("tanh", (False, True))
@pytest.mark.parametrize("dtype,pdtype", [(BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("hidden", (1, 3, 8, 24, 96, 255, 256, 264, 1000, 1111, 4096, 10008))
def test_without_records(taco, tanh, dtype, pdtype, hidden):
    for rows in (1, 5, 67):
        x, b = (2 * normal(hidden, rows, hidden)).to(dtype), normal(rows, hidden).to(pdtype)
        approximate = "tanh" if tanh else "none"
        check_value(taco.gelu(x, b, approximate=approximate, checkpoint=False).y, x.float() + b.float(), tanh)
        got = taco.gelu(x, approximate=approximate, checkpoint=False)
        check_value(got.y, x.float(), tanh)
        assert got.packed is None
