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
