"""GELU of infinities and NaN: the same in both forms, at every width, forward
and from records.  +infinity gives +infinity (slope 1), -infinity and NaN give
NaN; the largest finite numbers give 0 or themselves."""
import numpy as np
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


def same(got, want):
    return torch.equal(torch.nan_to_num(got.float().cpu(), nan=-7.0, posinf=7.0, neginf=-9.0),
                       torch.nan_to_num(torch.tensor(want), nan=-7.0, posinf=7.0, neginf=-9.0))


@pytest.mark.parametrize("approximate", ("none", "tanh"))
@pytest.mark.parametrize("dtype", (F32, BF16, F16))
@pytest.mark.parametrize("hidden", (64, 65))
def test_forward(taco, approximate, dtype, hidden):
    top = torch.finfo(dtype).max
    x = torch.zeros(3, hidden)
    x[1, :5] = torch.tensor([INF, -INF, NAN, top, -top])
    for bias in (None, torch.zeros(hidden, device="cuda")):
        y = taco.gelu(x.to(dtype).cuda(), bias, approximate=approximate, checkpoint=False).y
        assert same(y[1, :5], [INF, NAN, NAN, top, 0.0])
        assert not y[0].any() and not y[2].any() and not y[1, 5:].any()
    if hidden % 32 == 0:
        assert same(taco.gelu(x.to(dtype).cuda(), approximate=approximate, block=32).y[1, :5], [INF, NAN, NAN, top, 0.0])


@pytest.mark.parametrize("approximate", ("none", "tanh"))
@pytest.mark.parametrize("dtype", (F32, BF16, F16))
def test_from_records(taco, approximate, dtype):
    """E5M2 codes of infinities and a NaN, as records of another origin may hold, and the largest numbers."""
    record = np.zeros(40, np.uint8)
    record[:5] = 0x7C, 0xFC, 0x7E, 0x7B, 0xFB            # +inf, -inf, NaN, 57344, -57344
    record[32:] = np.array([1, 1], "<f4").view(np.uint8)
    g = taco.gelu_backward(torch.ones(1, 32, device="cuda", dtype=dtype), torch.from_numpy(record).cuda(),
                           approximate=approximate, block=32, code="e5m2", recompute=True)
    assert same(g.y[0, :5], [INF, NAN, NAN, 57344.0, 0.0])
    assert same(g.dx[0, :5], [1.0, NAN, NAN, 1.0, 0.0])
    assert not g.y[0, 5:].any()
    zeros = np.zeros(27)
    ref.within(g.dx[0, 5:], zeros + 0.5, ref.slope_bound(zeros), what="slope at 0")
