"""The gated layer's kernels with several tiles a CTA pair: accumulators and
buffers used again, and for dx whole tiles followed by ranges of K of the last
ones, whose sums go through the same buffers as the whole tiles' stores."""
import pytest
import torch

import gated_reference as gr
import training_reference as ref
from test_gpu_gated import BF16, F16, F32, check_backward, check_forward, taco, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,block,bias", [(BF16, 128, None), (F16, 64, F32), (BF16, 32, BF16), (BF16, None, F32)])
def test_many_tiles(taco, dtype, block, bias):  # noqa: F811
    """4 to 9 tiles a pair, the last row tile of 5000 rows ragged."""
    check_forward(taco, 5000, 72, 2048, dtype, "silu", bias, block)
    check_forward(taco, 2500, 200, 3968, dtype, "gelu", bias, block, "int8")


def test_input_gradient_whole_tiles_then_ranges(taco):  # noqa: F811
    """84 tiles on 76 pairs: eight of them cut into ranges of K."""
    check_backward(taco, 5376, 1024, 1024)
    check_backward(taco, 5300, 1001, 1024, F16)


def test_input_gradient_repeats(taco):  # noqa: F811
    """The same bits launch after launch, the next one's first tiles beside the last one's ranges."""
    rows, hidden, inner = 5376, 1024, 1024
    packed = ref.make_records(values(1, rows, 2 * inner), 32, "e4m3").cuda()
    dy, w = values(2, rows, inner).to(BF16).cuda(), (values(3, 2 * inner, hidden) / 32).to(BF16).cuda()
    first = taco.gated_linear_backward(dy, packed, w, block=32)
    for _ in range(20):
        again = taco.gated_linear_backward(dy, packed, w, block=32)
        assert torch.equal(first.dx, again.dx) and torch.equal(first.dz, again.dz)


def test_long_sums(taco):  # noqa: F811
    """K = 32768 along one accumulator."""
    x, w = values(1, 40, 32768).to(BF16), (values(2, 256, 32768) / 181).to(BF16)
    z, off = gr.product(ref.f64(x), ref.f64(w))
    y, off_y = gr.gated(z, off, "silu")
    ref.within(taco.gated_linear(x.cuda(), w.cuda()).y, y, off_y, what="few rows")
    ref.within(taco.gated_linear(x.cuda(), w.cuda(), checkpoint=True).y, y, off_y, what="pairs")


@pytest.mark.parametrize("rows", (65, 112, 128))
@pytest.mark.parametrize("inner", (12288, 12296, 12417))
def test_few_rows_at_the_last_width(taco, rows, inner):  # noqa: F811
    """Both sides of the width up to which 65 to 128 rows go to the few-row kernel."""
    check_forward(taco, rows, 72, inner, BF16, "silu", F32)


def test_few_rows_in_clusters(taco):  # noqa: F811
    """Every number of CTAs a cluster: 1 to 8 along K."""
    for inner in (30 * 64, 38 * 64, 45 * 64, 54 * 64, 68 * 64, 90 * 64, 136 * 64, 137 * 64, 280 * 64):
        check_forward(taco, 5, 2072, inner, F16, "gelu")


@pytest.mark.parametrize("rows,inner", [(200, 64), (200, 65), (300, 2432), (300, 2433), (300, 2400), (700, 1600), (2000, 576), (2000, 608),
                                        (256, 4864), (256, 4872), (257, 4864)])
@pytest.mark.parametrize("dtype,block", [(BF16, None), (F16, 64), (BF16, 32), (BF16, 128)])
def test_narrow_tiles(taco, rows, inner, dtype, block):  # noqa: F811
    """Both sides of the number of tiles up to which they are 64 columns wide."""
    if block is None or inner % block == 0:
        check_forward(taco, rows, 200, inner, dtype, "silu", F32 if rows % 3 else None, block, "e4m3" if rows % 7 else "int8")


def test_narrow_and_wide_tiles_agree(taco):  # noqa: F811
    """Either width adds the same products in the same order: records of blocks of 64 (narrow) and 128 (wide) aside, y is the same."""
    x, w = values(1, 300, 1000).to(BF16).cuda(), (values(2, 2 * 1280, 1000) / 32).to(BF16).cuda()
    narrow, wide = taco.gated_linear(x, w, checkpoint=True, block=64), taco.gated_linear(x, w, checkpoint=True, block=128)
    assert torch.equal(narrow.y, wide.y)
