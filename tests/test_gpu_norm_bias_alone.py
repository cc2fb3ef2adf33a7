"""The bias gradient of a layer norm without a weight: on every kernel's widths,
from x and from records, against 64 bits (training_reference's bound)."""
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
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("rows,hidden,records", [(1, 8, False), (5, 33, False), (301, 512, False), (40, 4097, False),
                                                 (9, 20480, False), (3, 20001, False), (301, 512, True), (9, 20480, True)])
@pytest.mark.parametrize("dtype,bias_dtype", [(BF16, F32), (F32, BF16), (F16, F16)])
def test_bias_gradient(taco, rows, hidden, dtype, bias_dtype, records):
    x, dy, bias = normal(1, rows, hidden).to(dtype).cuda(), normal(2, rows, hidden).to(dtype).cuda(), normal(3, hidden).to(bias_dtype).cuda()
    r = taco.layernorm(x, bias=bias, checkpoint=records, block=32)
    kept = {"packed": r.packed} if records else {"x": x, "mean": r.mean}
    g = taco.layernorm_backward(dy, r.rstd, block=32, bias_dtype=bias_dtype, **kept)
    assert g.dweight is None and g.dbias.dtype is bias_dtype
    d = ref.f64(dy)
    ref.within(g.dbias, d.sum(0), (rows + 16) * ref.U32 * np.abs(d).sum(0), what="dbias")
    # with a weight of ones the rows see the same arithmetic, the columns the same sums
    one = taco.layernorm_backward(dy, r.rstd, torch.ones_like(bias), block=32, **kept)
    assert torch.equal(g.dx, one.dx) and torch.equal(g.dbias, one.dbias)
    assert taco.layernorm_backward(dy, r.rstd, block=32, **kept).dbias is None
    assert taco.layernorm_backward(dy, r.rstd, block=32, bias_grad=False, bias_dtype=bias_dtype, **kept).dbias is None


def test_no_rows(taco):
    e = torch.empty(0, 96, device="cuda")
    r = taco.layernorm(e, bias=torch.ones(96, device="cuda"))
    g = taco.layernorm_backward(e, r.rstd, x=e, mean=r.mean, bias_dtype=BF16)
    assert g.dbias.shape == (96,) and not g.dbias.any() and g.dweight is None


def test_refusals(taco):
    x = normal(1, 4, 64).cuda()
    r = taco.layernorm(x)
    with pytest.raises(TypeError):
        taco.layernorm_backward(x, r.rstd, x=x, mean=r.mean, bias_dtype=torch.int8)
    with pytest.raises(TypeError):
        taco.layernorm_backward(x, r.rstd, torch.ones(64, device="cuda"), x=x, mean=r.mean, bias_dtype=BF16)
    same = taco.layernorm_backward(x, r.rstd, torch.ones(64, device="cuda"), x=x, mean=r.mean, bias_dtype=F32)
    assert torch.equal(same.dbias, taco.layernorm_backward(x, r.rstd, torch.ones(64, device="cuda"), x=x, mean=r.mean).dbias)
