"""The weight gradient's kernel over its launches and tiles: CTAs that leave
and are followed at once, pairs that take several tiles, long sums."""
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


@pytest.mark.parametrize("code,block", [("e4m3", 128), ("e5m2", 32), ("int8", 256)])
@pytest.mark.parametrize("rows,out,hidden,units", [
    (200, 2560, 2048, "80 whole tiles"),
    (1100, 2560, 2048, "76 whole tiles, 4 in two row ranges"),
    (2100, 5000, 2304, "152 whole tiles, 28 in two row ranges; 33 stages and three accumulators a tile"),
    (700, 4999, 1280, "100 whole tiles; rows of dY widened"),
])
def test_more_tiles_than_pairs(taco, rows, out, hidden, units, code, block):
    """Pairs that take several tiles: stages, teams and accumulators go on where
    the tile before left them.  Whole numbers, exact in every order: below 2^24."""
    dy, x = grid_values(rows, rows, out).cuda(), grid_values(out, rows, hidden).cuda()
    packed = taco.gelu(x, code=code, block=block).packed
    want = dy.t() @ x
    dy = dy.to(BF16)
    dw = taco.weight_grad(dy, packed, hidden, code=code, block=block)
    assert torch.equal(dw, want)
    scale, shift, before = (torch.randint(-3, 4, shape, generator=torch.Generator().manual_seed(i)).float().cuda()
                            for i, shape in enumerate(((hidden,), (hidden,), (out, hidden))))
    dy_sum = dy.float().sum(0)
    want = want * scale + dy_sum[:, None] * shift + before
    for dtype in (torch.float32, BF16):
        buffer = before.to(dtype, copy=True)
        taco.weight_grad(dy, packed, hidden, code=code, block=block, scale=scale, shift=shift, dy_sum=dy_sum, out=buffer,
                         accumulate=True)
        assert torch.equal(buffer, want.to(dtype))
    assert taco.device_status() == 0


@pytest.mark.parametrize("rows", (8192, 8257, 16384))
def test_long_sums(taco, rows):
    """76 tiles, all whole, over all rows.  A tensor-core accumulator cuts each
    addition by up to 2^-23 of its sum, 64 of them in 1024 rows, and the chunks'
    sums are added in rounded binary32: 192 + rows / 512 times 2^-24 of the terms'
    sizes at most, and in the 2-norm well below 1e-6, which one accumulator over
    all rows passes (3.2e-6)."""
    out, hidden = 19 * 256, 4 * 256
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy = (0.1 * torch.randn(rows, out, generator=g, device="cuda")).to(BF16)
    x = torch.randn(rows, hidden, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(hidden, generator=g, device="cuda"))
    packed = taco.gelu(x).packed
    x = taco.decompress(packed, rows, hidden, variant="ds_only").double()      # the records' values, exact in bf16
    want, size = dy.double().t() @ x, dy.double().abs().t() @ x.abs()
    off = (taco.weight_grad(dy, packed, hidden).double() - want).abs()
    assert bool((off <= (192 + rows / 512) * 2.0 ** -24 * size + 2.0 ** -24 * want.abs()).all())
    assert float(off.norm() / want.norm()) < 1e-6
