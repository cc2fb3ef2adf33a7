"""The training operators (layer norm, GELU, 8-bit checkpoints, weight
gradient) against plain implementations in 64 bits, at the sizes, types and
values where they can go wrong.  The bounds are training_reference.py's."""
import numpy as np
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CODES = ("e4m3", "e5m2", "int8")
EPS = 1e-5


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


def values(seed, *shape, scale=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * scale + mean


def params(seed, hidden, dtype):
    return (1 + 0.3 * values(seed, hidden)).to(dtype), (0.2 * values(seed + 1, hidden)).to(dtype)


# Rows and widths: one element, odd widths, widths of a vector, of a warp, of a CTA and their neighbours, wide rows.
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 255), (7, 256), (33, 1111), (64, 1024), (9, 2048), (17, 4096), (6, 5120),
          (5, 8192), (3, 8200), (3, 16384), (2, 20480), (2, 33000), (2, 40960), (700, 640), (1, 4096), (401, 96)]


def check_norm(taco, rows, hidden, dtype, pdtype, residual=False, block=None, code="e4m3", mean=0.4, affine=True):
    x = (values(rows + hidden, rows, hidden, mean=mean) * torch.exp(0.5 * values(3, hidden))).to(dtype)
    r = values(17, rows, hidden).to(dtype) if residual else None
    w, b = params(5, hidden, pdtype) if affine else (None, None)
    h = x if r is None else (x.float() + r.float()).to(dtype)
    cuda = lambda t: None if t is None else t.cuda()
    got = taco.layernorm(x.cuda(), cuda(w), cuda(b), eps=EPS, residual=cuda(r), checkpoint=block is not None,
                         block=block or 128, code=code)
    f = lambda t: None if t is None else ref.f64(t)
    y, mu, rstd, xhat, off_mu, off_rstd, off_xhat = ref.layernorm(ref.f64(h), f(w), f(b), EPS)
    wide = np.abs(f(w)) if affine else 1.0
    ref.within(got.mean, mu, off_mu, what="mean")
    ref.within(got.rstd, rstd, off_rstd, what="rstd")
    ref.within(got.y, y, wide * off_xhat + 4 * ref.U32 * (np.abs(xhat) * wide + (np.abs(f(b)) if affine else 0)), what="y")
    if residual:
        assert torch.equal(got.summed.cpu(), h)
    if block:
        q, alpha, s = ref.split(got.packed, block)
        assert np.all(alpha == 1)
        want = ref.scale_of(xhat, block, code)
        near = ref.scale_of(xhat + np.sign(xhat) * off_xhat, block, code), ref.scale_of(
            np.sign(xhat) * np.maximum(np.abs(xhat) - off_xhat, 0), block, code)
        assert np.all((s == want) | (s == near[0]) | (s == near[1]))
        val = ref.decode(got.packed, rows, hidden, block, code)
        half = ref.step_at(np.abs(xhat) + off_xhat, np.maximum(s, 0), block, code) / 2
        assert np.all(np.abs(val - xhat) <= half * (1 + 1e-12) + off_xhat)
        assert np.array_equal(ref.f64(taco.decompress(got.packed, rows, hidden, block, variant="ds_only", code=code)), val)
    return got


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, F32)])
def test_norm(taco, rows, hidden, dtype, pdtype):
    check_norm(taco, rows, hidden, dtype, pdtype)
    check_norm(taco, rows, hidden, dtype, pdtype, residual=True)


@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("hidden", (12288, 16376, 16384, 16383))
def test_norm_wide_rows_on_every_sm(taco, dtype, hidden):
    """More rows than SMs at the widest rows that registers hold: shared memory
    is full of rows and parameters."""
    block = 128 if hidden % 128 == 0 else None
    check_norm(taco, 170, hidden, dtype, F32, residual=True, block=block)
    check_norm(taco, 170, hidden, dtype, F32)
    check_norm_grad(taco, 170, hidden, dtype, F32, dsummed=True)
    check_norm_grad(taco, 170, hidden, dtype, F32, dsummed=True, block=block)


@pytest.mark.parametrize("affine,pdtype", [(False, F32), (True, BF16), (True, F16)])
def test_norm_parameters(taco, affine, pdtype):
    for hidden in (33, 1024, 4096):
        check_norm(taco, 12, hidden, BF16, pdtype, affine=affine)
        check_norm(taco, 12, hidden, F32, pdtype, affine=affine, residual=True)


def test_norm_weight_or_bias_alone(taco):
    x = values(1, 5, 512).cuda()
    w, b = (t.cuda() for t in params(2, 512, F32))
    plain = taco.layernorm(x).y
    assert torch.equal(taco.layernorm(x, weight=w).y, taco.layernorm(x, w, torch.zeros_like(b)).y)
    assert torch.equal(taco.layernorm(x, bias=b).y, taco.layernorm(x, torch.ones_like(w), b).y)
    assert torch.equal(plain, taco.layernorm(x, torch.ones_like(w), torch.zeros_like(b)).y)


@pytest.mark.parametrize("block", (32, 64, 128, 256, 512))
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", (BF16, F16, F32))
def test_norm_records(taco, block, code, dtype):
    for rows, hidden in ((1, block), (5, 3 * block), (19, 8 * block), (3, 2560), (2, 9216), (2, 34816)):
        if hidden % block == 0:
            check_norm(taco, rows, hidden, dtype, F32, block=block, code=code, residual=rows == 5)


def test_norm_large_mean(taco):
    """A mean 3000 times the deviation: the variance comes from centred values."""
    for hidden in (100, 4096, 16384):
        check_norm(taco, 8, hidden, F32, F32, mean=3000.0)


def test_norm_constant_rows(taco):
    """Zero variance: xhat = 0, y = bias, all-zero records."""
    for hidden in (1, 100, 512, 4096):
        x = torch.full((3, hidden), 2.5, device="cuda", dtype=BF16)
        w, b = (t.cuda() for t in params(4, hidden, F32))
        r = taco.layernorm(x, w, b, checkpoint=hidden % 128 == 0)
        assert torch.equal(r.y, b.to(BF16).expand(3, hidden))
        assert torch.all(r.mean == 2.5)
        assert torch.allclose(r.rstd, torch.full_like(r.rstd, EPS ** -0.5), rtol=4 * ref.U32)
        if r.packed is not None:
            q, alpha, s = ref.split(r.packed, 128)
            assert not q.any() and np.all(s == 0) and np.all(alpha == 1)


@pytest.mark.parametrize("hidden", (128, 333, 4096, 20480))
def test_norm_non_finite(taco, hidden):
    """NaN and infinities spoil their own row only, its records included."""
    x = values(9, 4, hidden)
    clean = taco.layernorm(x.cuda(), checkpoint=hidden % 128 == 0)
    x[1, hidden // 2] = float("nan")
    x[2, 0] = float("inf")
    r = taco.layernorm(x.cuda(), checkpoint=hidden % 128 == 0)
    assert torch.isnan(r.y[1]).all() and torch.isnan(r.y[2]).any()
    for row in (0, 3):
        assert torch.equal(r.y[row], clean.y[row])
    if r.packed is not None:
        v = taco.decompress(r.packed, 4, hidden, variant="ds_only")
        assert torch.isnan(v[1]).all() and torch.isnan(v[2]).any() and torch.isfinite(v[0]).all()


def check_norm_grad(taco, rows, hidden, dtype, pdtype, dsummed=False, block=None, code="e4m3", bias_grad=True, affine=True):
    x = (values(rows + hidden, rows, hidden, mean=0.3)).to(dtype)
    dy = values(7, rows, hidden, scale=0.1).to(dtype)
    if rows > 2:
        dy[1] = 0
    w = params(5, hidden, pdtype)[0] if affine else None
    ds = values(8, rows, hidden).to(dtype) if dsummed else None
    f = lambda t: None if t is None else ref.f64(t)
    mean = x.float().mean(1)
    rstd = torch.rsqrt((x.float() - mean[:, None]).square().mean(1) + EPS)
    cuda = lambda t: None if t is None else t.cuda()
    if block:
        packed = ref.make_records((x.float() - mean[:, None]) * rstd[:, None], block, code)
        xhat, off_xhat = ref.decode(packed, rows, hidden, block, code), 0.0
        kept = {"packed": packed.cuda()}
    else:
        xhat = (f(x) - f(mean)[:, None]) * f(rstd)[:, None]
        off_xhat = 2 * ref.U32 * (np.abs(xhat) + np.abs(f(mean) * f(rstd))[:, None])
        kept = {"x": x.cuda(), "mean": mean.cuda()}
    got = taco.layernorm_backward(dy.cuda(), rstd.cuda(), cuda(w), dsummed=cuda(ds), block=block or 128, code=code,
                                  bias_grad=bias_grad, **kept)
    dx, dw, db, off_dx, off_dw, off_db = ref.layernorm_grads(f(dy), xhat, f(rstd), f(w), off_xhat)
    if ds is not None:
        dx = dx + f(ds)
        off_dx = off_dx + 2 * ref.U32 * np.abs(f(ds))
    ref.within(got.dx, dx, off_dx, what="dx")
    if affine:
        ref.within(got.dweight, dw, off_dw, what="dweight")
    else:
        assert got.dweight is None and got.dbias is None
    if affine and bias_grad:
        ref.within(got.dbias, db, off_db, what="dbias")
    else:
        assert got.dbias is None


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, F32)])
def test_norm_grad(taco, rows, hidden, dtype, pdtype):
    check_norm_grad(taco, rows, hidden, dtype, pdtype)
    check_norm_grad(taco, rows, hidden, dtype, pdtype, dsummed=True)


@pytest.mark.parametrize("block", (32, 64, 128, 256, 512))
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", (BF16, F16, F32))
def test_norm_grad_records(taco, block, code, dtype):
    for rows, hidden in ((1, block), (5, 3 * block), (19, 8 * block), (400, 512), (3, 2560), (2, 9216), (2, 34816)):
        if hidden % block == 0:
            check_norm_grad(taco, rows, hidden, dtype, BF16, block=block, code=code, dsummed=rows == 5)


def test_norm_grad_options(taco):
    for hidden in (33, 1024):
        check_norm_grad(taco, 9, hidden, BF16, F32, bias_grad=False)
        check_norm_grad(taco, 9, hidden, F32, BF16, affine=False, dsummed=True)
        check_norm_grad(taco, 2000, hidden, F32, BF16)


def test_norm_gradient_against_differences(taco):
    """Directional derivatives of the 64-bit forward pass, central differences
    (h = 1e-5: truncation about h^2, rounding about 1e-16 / h)."""
    rows, hidden = 6, 384
    x, dy = values(1, rows, hidden), values(2, rows, hidden)
    w, b = params(3, hidden, F32)
    r = taco.layernorm(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    g = taco.layernorm_backward(dy.cuda(), r.rstd, w.cuda(), x=x.cuda(), mean=r.mean)
    loss = lambda X, W, B: float((ref.layernorm(X, W, B, EPS)[0] * ref.f64(dy)).sum())
    h, args = 1e-5, [ref.f64(x), ref.f64(w), ref.f64(b)]
    for i, grad in enumerate((g.dx, g.dweight, g.dbias)):
        v = ref.f64(values(10 + i, *args[i].shape))
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        slope = (loss(*up) - loss(*down)) / (2 * h)
        got = float((ref.f64(grad) * v).sum())
        size = np.abs(ref.f64(grad) * v).sum()
        assert abs(got - slope) <= 2e-5 * size + 1e-6, (i, got, slope)


@pytest.mark.parametrize("hidden", (96, 4096, 333))
def test_norm_no_rows(taco, hidden):
    e = torch.empty(0, hidden, device="cuda")
    w = torch.ones(hidden, device="cuda")
    r = taco.layernorm(e, w, w)
    assert r.y.shape == (0, hidden) and r.mean.shape == (0,)
    g = taco.layernorm_backward(e, r.rstd, w, x=e, mean=r.mean)
    assert g.dx.shape == (0, hidden) and not g.dweight.any() and not g.dbias.any()
    r = taco.layernorm(torch.empty(4, 0, device="cuda"))
    assert r.y.shape == (4, 0) and r.mean.shape == (4,)


# ---------------------------------------------------------------------------
# GELU
# ---------------------------------------------------------------------------

GELU_SHAPES = [(1, 32), (3, 64), (7, 544), (33, 1024), (2, 4096), (5, 20480), (300, 160)]


@pytest.mark.parametrize("tanh", (False, True))
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("block", (32, 64, 128, 256, 512))
def test_gelu(taco, tanh, code, dtype, pdtype, block):
    for rows, hidden in GELU_SHAPES:
        if hidden % block:
            continue
        x = values(rows, rows, hidden, scale=2.0).to(dtype)
        b = params(1, hidden, pdtype)[1] if rows % 2 else None
        u32 = x.float() + (0 if b is None else b.float())
        got = taco.gelu(x.cuda(), None if b is None else b.cuda(), approximate="tanh" if tanh else "none", block=block, code=code)
        u = ref.f64(u32)
        ref.within(got.y, ref.gelu(u, tanh)[0], ref.gelu_bound(u), what="y")
        val, s = ref.encode(u, block, code)          # u is a binary32 value: its record is exact
        q, alpha, gs = ref.split(got.packed, block)
        assert np.array_equal(gs, s) and np.all(alpha == 1)
        assert np.array_equal(ref.decode(got.packed, rows, hidden, block, code), val)


def test_gelu_without_records(taco):
    for hidden in (1, 7, 96, 1111, 4096):
        x = values(hidden, 5, hidden).to(BF16)
        b = params(1, hidden, BF16)[1]
        got = taco.gelu(x.cuda(), b.cuda(), checkpoint=False)
        u = ref.f64(x.float() + b.float())
        ref.within(got.y, ref.gelu(u, False)[0], ref.gelu_bound(u), what="y")
        assert got.packed is None


@pytest.mark.parametrize("tanh", (False, True))
def test_gelu_range(taco, tanh):
    """Every bf16 magnitude up to 2^56, both signs, and infinities' blocks."""
    bits = torch.arange(0, 0x5B80, dtype=torch.int32).to(torch.int16)
    x = torch.cat([bits.view(BF16), -bits.view(BF16)])
    x = torch.nn.functional.pad(x, (0, -x.numel() % 64)).view(-1, 64)
    got = taco.gelu(x.cuda(), approximate="tanh" if tanh else "none", block=32)
    u = ref.f64(x)
    ref.within(got.y, ref.gelu(u, tanh)[0], ref.gelu_bound(u), what="y")
    val, s = ref.encode(u, 32, "e4m3")
    assert np.array_equal(ref.decode(got.packed, *x.shape, 32, "e4m3"), val)
    g = taco.gelu_backward(torch.ones_like(x, dtype=F32).cuda(), got.packed, approximate="tanh" if tanh else "none",
                           block=32, recompute=True)
    y, slope = ref.gelu(val, tanh)
    ref.within(g.dx, slope, ref.slope_bound(val), what="dx")
    ref.within(g.y, y, ref.gelu_bound(val), what="y again")


def test_gelu_non_finite(taco):
    x = values(3, 4, 256)
    x[0, 3], x[1, 5], x[2, 200] = float("nan"), float("inf"), -float("inf")
    got = taco.gelu(x.cuda(), block=128)
    assert torch.isnan(got.y[0, 3]) and got.y[1, 5] == float("inf") and (got.y[2, 200] == 0 or torch.isnan(got.y[2, 200]))
    v = taco.decompress(got.packed, 4, 256, 128, variant="ds_only")
    bad = torch.isnan(v).view(4, 2, 128)
    want = torch.zeros(4, 2, dtype=torch.bool)
    want[0, 0] = want[1, 0] = want[2, 1] = True
    assert torch.equal(bad.all(-1).cpu(), want) and torch.equal(bad.any(-1).cpu(), want)
    g = taco.gelu_backward(torch.ones_like(x).cuda(), got.packed, block=128)
    assert torch.equal(torch.isnan(g.dx).view(4, 2, 128).all(-1).cpu(), want)


@pytest.mark.parametrize("tanh", (False, True))
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("block", (32, 128, 512))
def test_gelu_grad(taco, tanh, code, dtype, pdtype, block):
    for rows, hidden in GELU_SHAPES + [(1000, 512)]:
        if hidden % block:
            continue
        packed = ref.make_records(values(rows, rows, hidden, scale=1.5), block, code)
        u = ref.decode(packed, rows, hidden, block, code)
        dy = values(2, rows, hidden, scale=0.1).to(dtype)
        again = rows % 2 == 0
        got = taco.gelu_backward(dy.cuda(), packed.cuda(), approximate="tanh" if tanh else "none", bias_dtype=pdtype,
                                 recompute=again, block=block, code=code)
        y, slope = ref.gelu(u, tanh)
        d = ref.f64(dy)
        off = np.abs(d) * (ref.slope_bound(u) + ref.U32 * np.abs(slope))
        ref.within(got.dx, d * slope, off, what="dx")
        ref.within(got.dbias, (d * slope).sum(0), off.sum(0) + (rows + 16) * ref.U32 * np.abs(d * slope).sum(0), what="dbias")
        if again:
            ref.within(got.y, y, ref.gelu_bound(u), what="y")
        else:
            assert got.y is None
        if rows < 8:
            assert torch.equal(taco.gelu_backward(dy.cuda(), packed.cuda(), approximate="tanh" if tanh else "none",
                                                  block=block, code=code).dx, got.dx)


def test_gelu_gradient_against_differences(taco):
    u = values(1, 4, 256, scale=1.5)
    packed = ref.make_records(u, 64, "e4m3")
    v = ref.decode(packed, 4, 256, 64, "e4m3")
    for tanh in (False, True):
        g = taco.gelu_backward(torch.ones(4, 256).cuda(), packed.cuda(), approximate="tanh" if tanh else "none", block=64)
        h = 1e-5
        slope = (ref.gelu(v + h, tanh)[0] - ref.gelu(v - h, tanh)[0]) / (2 * h)
        assert np.max(np.abs(ref.f64(g.dx) - slope)) <= 2e-6 + 1e-8


def test_gelu_no_rows(taco):
    e = torch.empty(0, 256, device="cuda", dtype=BF16)
    r = taco.gelu(e)
    assert r.y.shape == (0, 256) and r.packed.numel() == 0
    g = taco.gelu_backward(e, r.packed, bias_dtype=F32, recompute=True)
    assert g.dx.shape == (0, 256) and not g.dbias.any() and g.y.shape == (0, 256)


# ---------------------------------------------------------------------------
# Weight gradient
# ---------------------------------------------------------------------------

def check_weight_grad(taco, rows, out, hidden, block=128, code="e4m3", dtype=F32, affine=None, accumulate=False, pow2=True):
    dy = values(1, rows, out, scale=0.1).to(BF16)
    u = values(2, rows, hidden) * torch.exp(0.5 * values(3, hidden))
    if pow2:
        packed = ref.make_records(u, block, code).cuda() if rows else torch.empty(0, dtype=torch.uint8, device="cuda")
    else:
        packed = taco.compress(u.to(BF16).cuda(), block, variant="ds_only", code=code)
    x = ref.decode(packed, rows, hidden, block, code)
    d = ref.f64(dy)
    want, size = d.T @ x, np.abs(d).T @ np.abs(x)
    # Products of bf16 values are exact.  Chunks of at most 1024 rows on the tensor cores: 64 + 16 additions, each cutting
    # at most 2^-23 of the running sum; the chunks' sums, or a plain chain over the rows, in rounded binary32 additions.
    off = max(96 * 2 + rows / 512, rows + 8) * ref.U32 * size
    if not pow2:
        off = off + 2.0 ** -8 * size                    # q s / alpha rounded to bf16 for the product
    scale = shift = dy_sum = None
    if affine is not None:
        scale, shift = params(4, hidden, affine)
        dy_sum = dy.float().sum(0)
        want = want * ref.f64(scale) + ref.f64(dy_sum)[:, None] * ref.f64(shift)
        off = off * np.abs(ref.f64(scale)) + 4 * ref.U32 * (np.abs(want) + np.abs(ref.f64(dy_sum)[:, None] * ref.f64(shift)))
    before = values(6, out, hidden).to(dtype)
    buffer = before.cuda() if accumulate else None
    if accumulate:
        want = want + ref.f64(before)
        off = off + 2 * ref.U32 * np.abs(want)
    cuda = lambda t: None if t is None else t.cuda()
    got = taco.weight_grad(dy.cuda(), packed, hidden, block=block, code=code, scale=cuda(scale), shift=cuda(shift),
                           dy_sum=cuda(dy_sum), out=buffer, accumulate=accumulate, dtype=dtype)
    assert buffer is None or got is buffer
    assert got.shape == (out, hidden) and got.dtype == dtype
    ref.within(got, want, off, what="dweight")
    assert taco.device_status() == 0


@pytest.mark.parametrize("rows", (1, 15, 16, 63, 64, 65, 200, 1030))
@pytest.mark.parametrize("out,hidden", [(8, 128), (1, 128), (127, 256), (128, 256), (136, 384), (256, 512), (264, 640), (520, 128)])
def test_weight_grad_shapes(taco, rows, out, hidden):
    check_weight_grad(taco, rows, out, hidden)


@pytest.mark.parametrize("block", (32, 64, 128, 256, 512))
@pytest.mark.parametrize("code", CODES)
def test_weight_grad_records(taco, block, code):
    for rows, out, hidden in ((70, 136, block), (200, 72, 3 * block), (333, 264, 2 * block), (64, 101, block)):
        check_weight_grad(taco, rows, out, hidden, block=block, code=code)
        check_weight_grad(taco, rows, out, hidden, block=block, code=code, pow2=False)


@pytest.mark.parametrize("dtype", (F32, BF16))
@pytest.mark.parametrize("affine", (None, F32, BF16, F16))
@pytest.mark.parametrize("accumulate", (False, True))
def test_weight_grad_epilogue(taco, dtype, affine, accumulate):
    for rows, out, hidden in ((100, 136, 384), (100, 99, 96), (3000, 64, 256), (700, 512, 1024)):
        check_weight_grad(taco, rows, out, hidden, block=32, dtype=dtype, affine=affine, accumulate=accumulate)


def test_weight_grad_long_and_wide(taco):
    check_weight_grad(taco, 9001, 128, 256)
    check_weight_grad(taco, 5000, 304, 1024, code="int8")
    check_weight_grad(taco, 600, 2056, 2048, block=512)
    check_weight_grad(taco, 4100, 7, 64, block=64)


def test_weight_grad_no_rows(taco):
    check_weight_grad(taco, 0, 136, 256)
    check_weight_grad(taco, 0, 136, 256, affine=F32)
    check_weight_grad(taco, 0, 40, 256, accumulate=True)
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    assert taco.weight_grad(torch.empty(4, 0, device="cuda", dtype=BF16), torch.zeros(4 * 136, dtype=torch.uint8, device="cuda"),
                            128).shape == (0, 128)
    assert taco.weight_grad(torch.empty(0, 4, device="cuda", dtype=BF16), empty, 0).shape == (4, 0)


def test_weight_grad_non_finite_block(taco):
    """A NaN block reaches its own columns only; a NaN gradient its own row."""
    u = values(1, 80, 256)
    u[3, 140] = float("inf")
    rec = taco.gelu(u.cuda(), block=64).packed
    dy = values(2, 80, 136).to(BF16)
    dw = taco.weight_grad(dy.cuda(), rec, 256, block=64)
    bad = torch.isnan(dw).cpu()
    assert bad[:, 128:192].all() and not bad[:, :128].any() and not bad[:, 192:].any()
    dy[7, 20] = float("nan")
    u[3, 140] = 0
    dw = taco.weight_grad(dy.cuda(), taco.gelu(u.cuda(), block=64).packed, 256, block=64)
    bad = torch.isnan(dw).cpu()
    assert bad[20].all() and not bad[:20].any() and not bad[21:].any()


def test_weight_grad_extreme_scales(taco):
    """Records whose scales reach the ends of the range (blocks of 2^-120 and of 2^50)."""
    u = values(1, 64, 256)
    u[:, :128] *= 2.0 ** -110
    u[:, 128:] *= 2.0 ** 50
    for code in CODES:
        packed = ref.make_records(u, 128, code)
        x = ref.decode(packed, 64, 256, 128, code)
        # bf16 subnormals (below 2^-126) lose bits of the smallest codes
        off_x = np.where(np.abs(x) < 2.0 ** -126, 2.0 ** -134, 0)
        dy = values(2, 64, 136, scale=1.0).to(BF16)
        got = taco.weight_grad(dy.cuda(), packed.cuda(), 256, code=code)
        d = ref.f64(dy)
        ref.within(got, d.T @ x, 200 * ref.U32 * (np.abs(d).T @ np.abs(x)) + np.abs(d).T @ off_x, what="dweight")


# ---------------------------------------------------------------------------
# Calls
# ---------------------------------------------------------------------------

def every_call(taco, x, w, b, dy, stream=None):
    hidden = x.shape[-1]
    r = taco.layernorm(x, w, b, checkpoint=True, residual=dy, stream=stream)
    g = taco.layernorm_backward(dy, r.rstd, w, packed=r.packed, dsummed=x, stream=stream)
    h = taco.layernorm_backward(dy, r.rstd, w, x=r.summed, mean=r.mean, stream=stream)
    u = taco.gelu(x, b, stream=stream)
    v = taco.gelu_backward(dy, u.packed, bias_dtype=F32, recompute=True, stream=stream)
    dw = taco.weight_grad(dy, r.packed, hidden, scale=w, shift=b, dy_sum=v.dbias, stream=stream)
    return [t for t in (*r, *g, *h, *u, *v, dw) if t is not None]


def inputs(rows=400, hidden=1024):
    w, b = (t.cuda() for t in params(3, hidden, F32))
    return values(1, rows, hidden).to(BF16).cuda(), w, b, values(2, rows, hidden).to(BF16).cuda()


@pytest.mark.parametrize("rows,hidden", [(400, 1024), (3, 256), (2100, 2048)])
def test_same_results_every_time(taco, rows, hidden):
    args = inputs(rows, hidden)
    first = every_call(taco, *args)
    for _ in range(3):
        for a, b in zip(first, every_call(taco, *args)):
            assert torch.equal(a, b)
    assert taco.device_status() == 0


def test_other_stream(taco):
    """On a stream of its own, behind work that is still running there, given
    as a stream or as a handle; workspaces freed early are not reused."""
    args = inputs()
    want = every_call(taco, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            late = [torch.empty_like(a) for a in args]
            for _ in range(8):
                busy @ busy
            for dst, src in zip(late, args):
                dst.copy_(src)
        got = every_call(taco, *late, stream=given)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_default_stream_as_a_number(taco):
    args = inputs(40, 512)
    want = every_call(taco, *args)
    torch.cuda.synchronize()
    for a, b in zip(want, every_call(taco, *args, stream=0)):
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    assert taco.device_status(device="cuda") == 0


def test_graph_capture(taco):
    args = inputs()
    want = every_call(taco, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = every_call(taco, *args)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_leading_dimensions(taco):
    x, w, b, dy = inputs(24, 512)
    flat = every_call(taco, x, w, b, dy)
    deep = every_call(taco, x.view(2, 3, 4, 512), w, b, dy.view(2, 3, 4, 512))
    for a, d in zip(flat, deep):
        assert torch.equal(a.reshape(-1), d.reshape(-1))


def test_refusals(taco):
    x, w, b, dy = inputs(8, 256)
    r = taco.layernorm(x, w, b, checkpoint=True)
    bad = pytest.raises
    with bad(TypeError):
        taco.layernorm(x.cpu(), w, b)
    with bad(TypeError):
        taco.layernorm(x.to(torch.int32))
    with bad(TypeError):
        taco.layernorm(x, w, b.to(BF16))                     # one type for weight and bias
    with bad(ValueError):
        taco.layernorm(x.t())                                # not contiguous
    with bad(ValueError):
        taco.layernorm(x, w[:128].contiguous(), b)
    with bad(ValueError):
        taco.layernorm(x, residual=dy[:4])
    with bad(taco.TacoError):
        taco.layernorm(x, eps=-1.0)
    with bad(taco.TacoError):
        taco.layernorm(x, checkpoint=True, block=96)
    with bad(taco.TacoError):
        taco.layernorm(x, checkpoint=True, block=512)        # hidden is no multiple of the block
    with bad(taco.TacoError) as e:
        taco.layernorm(x.reshape(-1)[1:513].view(2, 256))    # 2 bytes off a 16-byte boundary
    assert e.value.status == 4
    with bad(ValueError):
        taco.layernorm_backward(dy, r.rstd, w)
    with bad(ValueError):
        taco.layernorm_backward(dy, r.rstd, w, x=x, mean=r.mean, packed=r.packed)
    with bad(ValueError):
        taco.layernorm_backward(dy, r.rstd, w, packed=r.packed[:-8].contiguous())
    with bad(TypeError):
        taco.layernorm_backward(dy, r.rstd.to(BF16), w, x=x, mean=r.mean)
    with bad(ValueError):
        taco.gelu(x, approximate="fast")
    with bad(TypeError):
        taco.gelu_backward(dy, r.packed, bias_dtype=torch.int8)
    with bad(TypeError):
        taco.weight_grad(dy.float(), r.packed, 256)
    with bad(ValueError):
        taco.weight_grad(dy, r.packed, 256, shift=b)
    with bad(ValueError):
        taco.weight_grad(dy, r.packed, 256, accumulate=True)
    with bad(TypeError):
        taco.weight_grad(dy, r.packed, 256, dtype=F16)
    with bad(ValueError):
        taco.weight_grad(dy, r.packed, 256, out=torch.empty(256, 128, device="cuda"))
    with bad(ValueError):
        taco.weight_grad(dy, r.packed, 128)
    with bad(KeyError):
        taco.gelu(x, code="e3m4")


def test_overlap_refused(taco):
    """An output on an input is refused before anything is launched."""
    from fp8_compression_tensor_gb300 import _training as t
    import ctypes
    x = values(1, 8, 256).to(BF16).cuda()
    keep = x.clone()
    stats = torch.zeros(64, device="cuda")
    lib = t._library()
    args = t._LayerNormArgs(x.data_ptr(), None, None, None, x.data_ptr(), None, stats.data_ptr(), stats.data_ptr() + 128, None,
                            8, 256, EPS, 0, 2, 128, 0)
    assert lib.taco_layernorm(ctypes.byref(args), None) == 6
    args = t._GeluArgs(x.data_ptr(), None, x.data_ptr() + 512, None, 8, 256, 0, 2, 0, 128, 0)
    assert lib.taco_gelu(ctypes.byref(args), None) == 6
    torch.cuda.synchronize()
    assert torch.equal(x, keep) and not stats.any()
