"""The RMS norm of rows whose squares leave binary32: the sum of squares overflows
from about 2^64 on and underflows, where eps is as small, below 2^-63.  The bounds
are those of gated_reference.py; scales are chosen so that rstd is no subnormal
number."""
import numpy as np
import pytest
import torch

import gated_reference as gr
import training_reference as ref
from test_gpu_rmsnorm import BF16, EPS, F16, F32, check_records, cuda, taco, values  # noqa: F401

pytestmark = pytest.mark.gpu

# A warp, several warps, rows that start anywhere, the widest rows in registers, rows read twice, and odd ones of these.
WIDTHS = (128, 333, 512, 4096, 8200, 16383, 20480, 30208, 33001)


def check(taco, x, weight, eps, residual=None, records=False):
    rows, hidden = x.shape
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    assert torch.isfinite(h).all()
    got = taco.rmsnorm(x.cuda(), cuda(weight), eps=eps, residual=cuda(residual), checkpoint=records)
    y, rstd, xhat, off_rstd, off_xhat = gr.rmsnorm(ref.f64(h), None if weight is None else ref.f64(weight), eps)
    off_y = (1 if weight is None else np.abs(ref.f64(weight))) * off_xhat + 2 * ref.U32 * np.abs(y)
    ref.within(got.rstd, rstd, off_rstd, what="rstd")
    ref.within(got.y, y, off_y, what="y")
    if residual is not None:
        assert torch.equal(got.summed.cpu(), h)
    if records:
        check_records(got.packed, xhat, off_xhat, rows, hidden, 128, "e4m3")
        both = taco.rmsnorm(x.cuda(), cuda(weight), eps=eps, residual=cuda(residual), checkpoint=True, packed_y=True)
        assert torch.equal(both.packed, got.packed)
        check_records(both.y, y, off_y, rows, hidden, 128, "e4m3")
    return got


@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("power", (61, 64, 100, 120))
def test_large_rows(taco, hidden, dtype, power):  # noqa: F811
    x, w = values(1, 3, hidden).to(dtype) * 2.0 ** power, 1 + 0.3 * values(2, hidden)
    check(taco, x, w, EPS, records=hidden % 128 == 0)
    check(taco, x, None, 0.0, residual=(values(3, 3, hidden) * 2.0 ** power).to(dtype))


@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("power", (-45, -64, -80, -100))
def test_small_rows(taco, hidden, dtype, power):  # noqa: F811
    """With eps below the squares, of their size and above them, and without eps."""
    x, w = values(1, 3, hidden).to(dtype) * 2.0 ** power, 1 + 0.3 * values(2, hidden)
    for eps in (0.0, max(2.0 ** (2 * power - 3), 2.0 ** -126), max(2.0 ** (2 * power), 2.0 ** -120), 2.0 ** -70, EPS):
        check(taco, x, w, eps, records=hidden % 128 == 0)


@pytest.mark.parametrize("hidden", (1, 7, 64, 1001, 20481))
def test_one_large_element(taco, hidden):  # noqa: F811
    x = torch.zeros(2, hidden)
    x[0, hidden // 2], x[1, 0] = 3e38, -2.0 ** 70
    check(taco, x, None, EPS)
    check(taco, x.to(BF16), None, 0.0)


@pytest.mark.parametrize("rows,hidden", [(5, 640), (700, 640), (401, 97), (170, 4099), (9, 30208), (9, 33001)])
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_neighbours_keep_their_bits(taco, rows, hidden, dtype):  # noqa: F811
    """Rows between such rows are what they are alone, and the large rows are the same from run to run."""
    x = values(4, rows, hidden).to(dtype)
    plain = taco.rmsnorm(x.cuda(), eps=0.0)
    mixed = x.clone()
    mixed[::3] *= 2.0 ** 90
    mixed[1::3] *= 2.0 ** -90
    got = taco.rmsnorm(mixed.cuda(), eps=0.0)
    assert torch.equal(got.y[2::3], plain.y[2::3]) and torch.equal(got.rstd[2::3], plain.rstd[2::3])
    y, rstd, _, off_rstd, off_xhat = gr.rmsnorm(ref.f64(mixed), None, 0.0)
    ref.within(got.rstd, rstd, off_rstd, what="rstd")
    ref.within(got.y, y, off_xhat + 2 * ref.U32 * np.abs(y), what="y")
    assert torch.equal(got.y, taco.rmsnorm(mixed.cuda(), eps=0.0).y)


@pytest.mark.parametrize("hidden", (128, 333, 4096, 20480, 33001))
def test_what_stays_outside(taco, hidden):  # noqa: F811
    """An infinity still makes its row zeros but for itself (NaN), a NaN spoils its row, and a row of zeros has no
    norm without eps."""
    x = values(9, 4, hidden) * 2.0 ** 80
    x[0, hidden // 2], x[1, 0], x[2] = float("inf"), float("nan"), 0.0
    r = taco.rmsnorm(x.cuda(), eps=0.0)
    y = r.y.cpu()
    assert torch.isnan(y[0, hidden // 2]) and int(torch.count_nonzero(y[0])) == 1 and r.rstd[0] == 0
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and torch.isinf(r.rstd[2])
    assert torch.isfinite(y[3]).all() and abs(float(y[3].double().square().mean()) - 1) < 1e-4
    assert not taco.rmsnorm(x[2:3].cuda()).y.any()


@pytest.mark.parametrize("hidden", (128, 333, 4096, 30208, 33001))
@pytest.mark.parametrize("power", (-100, -60, -40, 40, 64, 100))
def test_gradient(taco, hidden, power):  # noqa: F811
    """The gradient from such rows and the rstd that the norm returns for them, where a x stays in binary32."""
    x, dy = values(1, 4, hidden) * 2.0 ** power, values(2, 4, hidden)
    w = 1 + 0.3 * values(3, hidden)
    rstd = taco.rmsnorm(x.cuda(), eps=0.0).rstd
    got = taco.rmsnorm_backward(dy.cuda(), rstd, w.cuda(), x=x.cuda())
    r64 = ref.f64(rstd)
    xhat = ref.f64(x) * r64[:, None]
    dx, dw, off_dx, off_dw = gr.rmsnorm_grads(ref.f64(dy), xhat, r64, ref.f64(w), ref.U32 * np.abs(xhat))
    ref.within(got.dx, dx, off_dx, what="dx")
    ref.within(got.dweight, dw, off_dw, what="dweight")
