"""The training operators on empty tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


@pytest.mark.parametrize("stream", (False, True))
def test_statistics_of_rows_without_elements(taco, stream):
    """NaN, whatever the memory held before."""
    side = torch.cuda.Stream() if stream else None
    for dirty in (3.0, 7.0):
        with torch.cuda.stream(side):
            held = [torch.full((5,), dirty, device="cuda") for _ in range(4)]
            del held
        torch.cuda.synchronize()
        r = taco.layernorm(torch.empty(5, 0, device="cuda"), stream=side)
        torch.cuda.synchronize()
        assert r.y.shape == (5, 0) and r.mean.shape == (5,) and r.rstd.shape == (5,)
        assert torch.isnan(r.mean).all() and torch.isnan(r.rstd).all()


def test_norm_gradient_of_rows_without_elements(taco):
    e, w = torch.empty(5, 0, device="cuda"), torch.empty(0, device="cuda")
    r = taco.layernorm(e, w, w, residual=e)
    g = taco.layernorm_backward(e, r.rstd, w, x=r.summed, mean=r.mean, dsummed=e)
    assert g.dx.shape == (5, 0) and g.dweight.shape == (0,) and g.dbias.shape == (0,)
    r = taco.layernorm(e, checkpoint=True)
    assert taco.layernorm_backward(e, r.rstd, packed=r.packed).dx.shape == (5, 0)


@pytest.mark.parametrize("rows,out,hidden", [(4, 0, 128), (4, 8, 0), (0, 0, 128), (0, 8, 0), (4, 0, 0)])
def test_weight_gradient_without_elements(taco, rows, out, hidden):
    dy = torch.zeros(rows, out, device="cuda", dtype=BF16)
    packed = torch.zeros(taco.compressed_bytes(rows, hidden, 128), dtype=torch.uint8, device="cuda")
    param = torch.ones(hidden, device="cuda")
    dw = taco.weight_grad(dy, packed, hidden, scale=param, shift=param, dy_sum=torch.zeros(out, device="cuda"))
    assert dw.shape == (out, hidden) and dw.dtype is F32


@pytest.mark.parametrize("approximate", ("none", "tanh"))
def test_gelu_of_rows_without_elements(taco, approximate):
    e = torch.empty(5, 0, device="cuda", dtype=BF16)
    r = taco.gelu(e, torch.empty(0, device="cuda"), approximate=approximate)
    g = taco.gelu_backward(e, r.packed, approximate=approximate, bias_dtype=F32, recompute=True)
    assert r.y.shape == g.dx.shape == g.y.shape == (5, 0) and g.dbias.shape == (0,)
