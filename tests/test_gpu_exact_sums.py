"""The gated layer's products on inputs whose sums are exact (exact_sums.py): the
outputs have to be equal, bit by bit, at sums up to the longest, at many tiles a
pair of CTAs, and beyond 32-bit offsets; and the RMS norm and its gradient beyond
32-bit offsets."""
import pytest
import torch

import exact_sums as ex
import training_reference as ref
from test_gpu_gated import BF16, F16, F32, taco  # noqa: F401

pytestmark = pytest.mark.gpu


def check_layer(taco, rows, hidden, inner, dtype, block=None, code="e4m3", keep=None):
    x, w, bias = ex.layer(rows, hidden, inner, device="cuda")
    z, y = ex.layer_values(x, w, bias)
    got = taco.gated_linear(x.to(dtype), w.to(dtype), bias, checkpoint=block is not None, block=block or 128, code=code)
    assert torch.equal(got.y, y.to(dtype))
    if block:
        rows_seen = slice(None) if keep is None else keep
        packed = got.packed.view(rows, -1)[rows_seen].reshape(-1).cpu()
        assert torch.equal(packed, ref.make_records(z[rows_seen].cpu(), block, code))


# Few rows: a CTA a tile (137 tiles of 64 columns on), clusters of eight along K, the most tokens, an odd width.
@pytest.mark.parametrize("rows,hidden,inner", [(5, 32768, 8768), (40, 32768, 128), (128, 16384, 256), (17, 32761, 96), (64, 8200, 3456),
                                               (1, 32768, 17600)])
@pytest.mark.parametrize("dtype", (BF16, F16))
def test_few_rows(taco, rows, hidden, inner, dtype):  # noqa: F811
    check_layer(taco, rows, hidden, inner, dtype)


@pytest.mark.parametrize("rows,hidden,inner,block", [(200, 32768, 64, None), (200, 32768, 64, 64), (300, 32768, 256, 128), (300, 32765, 256, 32),
                                                     (40, 32768, 160, 32), (256, 4096, 4864, None), (257, 4096, 4864, None)])
@pytest.mark.parametrize("dtype", (BF16, F16))
def test_pairs(taco, rows, hidden, inner, block, dtype):  # noqa: F811
    check_layer(taco, rows, hidden, inner, dtype, block)


@pytest.mark.parametrize("dtype,block,code", [(BF16, None, "e4m3"), (F16, 128, "e4m3"), (BF16, 32, "int8"), (BF16, 64, "e5m2")])
def test_many_tiles_a_pair(taco, dtype, block, code):  # noqa: F811
    """640 tiles on 76 pairs, eight or nine each, the last row tile ragged."""
    rows = 5000
    keep = torch.cat([torch.arange(0, rows, 37), torch.arange(rows - 8, rows)])
    check_layer(taco, rows, 72, 4096, dtype, block, code, keep)


@pytest.mark.parametrize("block", (None, 32))
def test_longest_sum(taco, block):  # noqa: F811
    """2^24 terms: of few rows in a cluster of eight, with records in one pair's accumulator."""
    check_layer(taco, 3, 1 << 24, 32, BF16, block)


def check_gradient(taco, rows, hidden, inner, dtype, block=32, code="e4m3"):
    dy, up, w = ex.gradient(rows, hidden, inner, device="cuda")
    packed = ref.make_records(torch.cat([torch.full_like(up, 32), up], 1).float().cpu(), block, code).cuda()
    dz, dx, db = ex.gradient_values(dy, up, w)
    got = taco.gated_linear_backward(dy.to(dtype), packed, w.to(dtype), bias_dtype=F32, recompute=True, block=block, code=code)
    assert torch.equal(got.dz, dz.to(dtype)) and torch.equal(got.y, (32 * up).to(dtype))
    assert torch.equal(got.dx, dx.to(dtype)) and torch.equal(got.dbias, db)


# Long sums, the last wave's tiles cut into ranges of K, whole tiles before them, tiles that are all whole, odd widths.
@pytest.mark.parametrize("rows,hidden,inner", [(130, 200, 16384), (257, 1024, 2752), (1, 8, 32), (1000, 2048, 1024), (5376, 1024, 256),
                                               (300, 1001, 4096), (640, 5120, 512)])
@pytest.mark.parametrize("dtype", (BF16, F16))
def test_input_gradient(taco, rows, hidden, inner, dtype):  # noqa: F811
    check_gradient(taco, rows, hidden, inner, dtype)


def test_input_gradient_longest_sum(taco):  # noqa: F811
    """2 inner = 2^24 with one row: -1, 0 and 1 from SiLU's 32 would pass 2^24, so few of them are not 0."""
    inner, hidden = 1 << 23, 16
    dy, up = ex.signs(1, 1, inner, density=2.0 ** -8, device="cuda"), ex.signs(2, 1, inner, device="cuda")
    w = ex.signs(3, 2 * inner, hidden, device="cuda")
    records = torch.empty(2, inner // 128, 136, dtype=torch.uint8, device="cuda")
    records[:, :, 128:132] = torch.tensor([1.0]).view(torch.uint8).cuda()
    records[0, :, 132:] = torch.tensor([32.0 / 256]).view(torch.uint8).cuda()
    records[1, :, 132:] = torch.tensor([1.0 / 256]).view(torch.uint8).cuda()
    records[0, :, :128] = 0x78                                                    # 256 in E4M3
    records[1, :, :128] = torch.where(up.view(-1, 128) < 0, 0xf8, 0x78).to(torch.uint8)
    got = taco.gated_linear_backward(dy.to(BF16), records.view(-1), w.to(BF16))
    dz = torch.cat([dy * up, 32 * dy], 1).float()
    assert torch.equal(got.dz, dz.to(BF16))
    assert float((dz.abs()).sum()) < 2 ** 24
    assert torch.equal(got.dx, (dz @ w.float()).to(BF16))


def test_offsets_beyond_32_bits(taco):  # noqa: F811
    """The last rows of tensors of more than 2^31 elements are what they are alone."""
    rows, hidden, inner, tail = 140_000, 64, 16384, 300
    x, w, bias = ex.layer(rows, hidden, inner, device="cuda")
    x, w = x.to(BF16), w.to(BF16)
    whole, last = taco.gated_linear(x, w, bias, checkpoint=True), taco.gated_linear(x[-tail:].clone(), w, bias, checkpoint=True)
    assert torch.equal(whole.y[-tail:], last.y)
    assert torch.equal(whole.packed.view(rows, -1)[-tail:], last.packed.view(tail, -1))
    del whole, x
    dy = ex.signs(5, rows, inner, device="cuda").to(BF16)
    # z_gate = 32 and z_up = 1 throughout
    records = torch.full((rows, 2, inner // 128, 136), 0x78, dtype=torch.uint8, device="cuda")
    records[..., 128:132] = torch.tensor([1.0]).view(torch.uint8).cuda()
    records[:, 0, :, 132:] = torch.tensor([32.0 / 256]).view(torch.uint8).cuda()
    records[:, 1, :, 132:] = torch.tensor([1.0 / 256]).view(torch.uint8).cuda()
    got = taco.gated_linear_backward(dy, records.view(-1), w, bias_dtype=F32, recompute=True)
    last = dy[-tail:].float()
    dz = torch.cat([last, 32 * last], 1)
    assert torch.equal(got.dz[-tail:], dz.to(BF16)) and torch.equal(got.dx[-tail:], (dz @ w.float()).to(BF16))
    assert bool((got.y[-tail:] == 32).all())
    sums = sum(part.float().sum(0) for part in dy.split(10_000))
    assert torch.equal(got.dbias, torch.cat([sums, 32 * sums]))


@pytest.mark.parametrize("rows,hidden", [(530_000, 4096), (530_001, 4099), (72_000, 30208)])
def test_norm_offsets_beyond_32_bits(taco, rows, hidden):  # noqa: F811
    x, dy = ex.signs(1, rows, hidden, device="cuda").to(BF16), ex.signs(2, rows, hidden, density=0.5, device="cuda").to(BF16)
    w, tail = torch.ones(hidden, device="cuda"), 301
    sub = [t[-tail:].clone() for t in (x, dy)]   # (a view may lie where calls refuse it)
    records = hidden % 128 == 0
    whole, last = (taco.rmsnorm(a, w, residual=b, checkpoint=records) for a, b in ((x, dy), sub))
    for a, b in ((whole.y, last.y), (whole.rstd, last.rstd), (whole.summed, last.summed)):
        assert torch.equal(a[-tail:], b)
    if records:
        assert torch.equal(whole.packed.view(rows, -1)[-tail:], last.packed.view(tail, -1))
    del whole
    one = torch.ones(rows, device="cuda")
    whole, last = taco.rmsnorm_backward(dy, one, w, x=x), taco.rmsnorm_backward(sub[1], one[:tail], w, x=sub[0])
    assert torch.equal(whole.dx[-tail:], last.dx)
    sums = sum((a.float() * b.float()).sum(0) for a, b in zip(dy.split(10_000), x.split(10_000)))   # whole numbers below 2^24
    assert torch.equal(whole.dweight, sums)
