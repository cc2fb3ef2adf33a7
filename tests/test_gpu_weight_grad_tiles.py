"""The weight gradient's kernel over its launches and tiles: CTAs that leave
and are followed at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


def grid_values(seed, *shape):
    """Whole numbers in -8 .. 8, which the records hold exactly."""
    return torch.randint(-8, 9, shape, generator=torch.Generator().manual_seed(seed)).float()


def test_short_launches_back_to_back(taco):
    """Launches of a stage or a few, where a CTA leaves right behind its last
    products, each followed at once by one that takes its shared memory: sums
    of whole numbers, exact in every order."""
    cases = []
    for i, (rows, out, hidden) in enumerate([(1, 8, 128), (64, 256, 256), (65, 136, 384), (300, 520, 1024), (200, 101, 640)]):
        dy, x = grid_values(i, rows, out), grid_values(10 + i, rows, hidden)
        packed = taco.gelu(x.cuda(), code="int8").packed            # records of x
        assert torch.equal(taco.decompress(packed, rows, hidden, variant="ds_only", code="int8").float().cpu(), x)
        cases.append((dy.to(BF16).cuda(), packed, hidden, (dy.t() @ x).cuda()))
    got = []
    for turn in range(60):
        for j, (dy, packed, hidden, _) in enumerate(cases):
            got.append((j, taco.weight_grad(dy, packed, hidden, code="int8")))
    assert taco.device_status() == 0
    for j, dw in got:
        assert torch.equal(dw, cases[j][3])
