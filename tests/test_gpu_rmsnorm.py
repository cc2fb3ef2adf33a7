"""The RMS norm and its gradient against plain implementations in 64 bits, at the
sizes, types and values where they can go wrong.  The bounds are those of
gated_reference.py."""
import ctypes

import numpy as np
import pytest
import torch

import gated_reference as gr
import training_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CODES = ("e4m3", "e5m2", "int8")
EPS = 1e-6


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


def values(seed, *shape, scale=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * scale + mean


def cuda(t):
    return None if t is None else t.cuda()


# One element, odd widths, widths of a vector, a warp, a CTA and their neighbours, wide rows; more rows than SMs.
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 255), (7, 256), (33, 1111), (64, 1024), (9, 2048), (17, 4096), (6, 5120), (5, 8192),
          (3, 8200), (3, 16384), (2, 16383), (2, 20480), (2, 33001), (2, 40960), (700, 640), (1, 4096), (401, 97), (1300, 33),
          (170, 4099), (200, 2), (333, 9)]


def check_records(packed, want, off, rows, hidden, block, code):
    """Records hold `want` up to half a step of their grid, with a scale that
    the bound `off` on the values allows."""
    q, alpha, s = ref.split(packed, block)
    assert np.all(alpha == 1)
    near = [ref.scale_of(want, block, code), ref.scale_of(np.abs(want) + off, block, code),
            ref.scale_of(np.maximum(np.abs(want) - off, 0), block, code)]
    assert np.all((s == near[0]) | (s == near[1]) | (s == near[2]))
    val = ref.decode(packed, rows, hidden, block, code)
    half = ref.step_at(np.abs(want) + off, s, block, code) / 2
    assert np.all(np.abs(val - want) <= half * (1 + 1e-12) + off)
    return val


def check_norm(taco, rows, hidden, dtype, pdtype, residual=False, block=None, code="e4m3", affine=True, packed_y=False):
    x = (values(rows + hidden, rows, hidden, mean=0.1) * torch.exp(0.5 * values(3, hidden))).to(dtype)
    r = values(17, rows, hidden).to(dtype) if residual else None
    w = (1 + 0.3 * values(5, hidden)).to(pdtype) if affine else None
    h = x if r is None else (x.float() + r.float()).to(dtype)
    got = taco.rmsnorm(x.cuda(), cuda(w), eps=EPS, residual=cuda(r), checkpoint=block is not None, packed_y=packed_y,
                       block=block or 128, code=code)
    y, rstd, xhat, off_rstd, off_xhat = gr.rmsnorm(ref.f64(h), ref.f64(w) if affine else None, EPS)
    wide = np.abs(ref.f64(w)) if affine else 1.0
    off_y = wide * off_xhat + 2 * ref.U32 * np.abs(y)
    ref.within(got.rstd, rstd, off_rstd, what="rstd")
    if packed_y:
        val = check_records(got.y, y, off_y, rows, hidden, block, code)
        assert np.array_equal(ref.f64(taco.decompress(got.y, rows, hidden, block, variant="ds_only", code=code)), val)
    else:
        ref.within(got.y, y, off_y, what="y")
    assert (got.summed is None) == (r is None) and (r is None or torch.equal(got.summed.cpu(), h))
    if block:
        check_records(got.packed, xhat, off_xhat, rows, hidden, block, code)
    return got


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, F32), (BF16, BF16)])
def test_norm(taco, rows, hidden, dtype, pdtype):
    check_norm(taco, rows, hidden, dtype, pdtype)
    check_norm(taco, rows, hidden, dtype, pdtype, residual=True)
    check_norm(taco, rows, hidden, dtype, pdtype, affine=False)


@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("hidden", (7176, 12288, 16376, 16384, 16383, 16377))
def test_wide_rows_on_every_sm(taco, dtype, hidden):
    """More rows than SMs at the widest rows that shared memory holds."""
    block = 128 if hidden % 128 == 0 else None
    check_norm(taco, 170, hidden, dtype, F32, residual=True, block=block)
    check_norm(taco, 170, hidden, dtype, F32)
    check_grad(taco, 170, hidden, dtype, F32, dsummed=True)
    check_grad(taco, 170, hidden, dtype, F32, dsummed=True, block=block)


@pytest.mark.parametrize("block", (32, 64, 128, 256, 512))
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", (BF16, F16, F32))
def test_records(taco, block, code, dtype):
    for rows, hidden in ((1, block), (5, 3 * block), (19, 8 * block), (3, 2560), (2, 9216), (2, 34816), (310, 512)):
        if hidden % block == 0:
            check_norm(taco, rows, hidden, dtype, F32, block=block, code=code, residual=rows == 5, packed_y=rows % 2 == 1)


def test_packed_output_alone(taco):
    x = values(4, 6, 1024).to(BF16).cuda()
    w = (1 + 0.1 * values(5, 1024)).cuda()
    both = taco.rmsnorm(x, w, checkpoint=True, packed_y=True)
    alone = taco.rmsnorm(x, w, packed_y=True)
    assert alone.packed is None and torch.equal(alone.y, both.y)
    assert torch.equal(taco.rmsnorm(x, w, checkpoint=True).packed, both.packed)
    assert torch.equal(taco.rmsnorm(x, packed_y=True).y, both.packed)   # without a weight y is xhat


@pytest.mark.parametrize("hidden", (128, 333, 4096, 20480))
def test_non_finite(taco, hidden):
    """NaN and infinities spoil their own row only, its records included."""
    x = values(9, 4, hidden)
    clean = taco.rmsnorm(x.cuda(), checkpoint=hidden % 128 == 0)
    x[1, hidden // 2] = float("nan")
    x[2, 0] = float("inf")
    r = taco.rmsnorm(x.cuda(), checkpoint=hidden % 128 == 0)
    assert torch.isnan(r.y[1]).all() and torch.isnan(r.y[2, 0]) and torch.all(r.y[2, 1:] == 0)
    for row in (0, 3):
        assert torch.equal(r.y[row], clean.y[row])
    if r.packed is not None:
        values_ = taco.decompress(r.packed, 4, hidden, variant="ds_only")
        assert torch.isnan(values_[1]).all() and torch.isnan(values_[2, :128]).all()


def test_zero_rows_and_empty(taco):
    for hidden in (1, 100, 512, 4096, 20480):
        x = torch.zeros(3, hidden, device="cuda", dtype=BF16)
        r = taco.rmsnorm(x, torch.ones(hidden, device="cuda"), eps=EPS, checkpoint=hidden % 128 == 0)
        assert not r.y.any() and torch.allclose(r.rstd, torch.full_like(r.rstd, EPS ** -0.5), rtol=4 * ref.U32)
        if r.packed is not None:
            q, alpha, s = ref.split(r.packed, 128)
            assert not q.any() and np.all(s == 0) and np.all(alpha == 1)
    w = torch.ones(256, device="cuda")
    r = taco.rmsnorm(torch.empty(0, 256, device="cuda", dtype=BF16), w, checkpoint=True)
    assert r.y.shape == (0, 256) and r.rstd.shape == (0,) and r.packed.numel() == 0
    g = taco.rmsnorm_backward(r.y, r.rstd, w, packed=r.packed)
    assert g.dx.shape == (0, 256) and not g.dweight.any()
    r = taco.rmsnorm(torch.empty(3, 0, device="cuda", dtype=BF16))
    assert r.y.shape == (3, 0) and torch.isnan(r.rstd).all()


def check_grad(taco, rows, hidden, dtype, pdtype, dsummed=False, block=None, code="e4m3", affine=True):
    x = (values(rows + hidden + 1, rows, hidden) * torch.exp(0.4 * values(3, hidden))).to(dtype)
    dy, ds = values(8, rows, hidden, scale=0.1).to(dtype), values(9, rows, hidden, scale=0.1).to(dtype) if dsummed else None
    w = (1 + 0.3 * values(5, hidden)).to(pdtype) if affine else None
    rstd = torch.rsqrt(x.float().square().mean(1) + EPS)
    r64 = ref.f64(rstd)
    if block:
        packed = ref.make_records(x.float() * rstd[:, None], block, code)
        xhat, off_xhat, source = ref.decode(packed, rows, hidden, block, code), 0.0, dict(packed=packed.cuda())
    else:
        xhat = ref.f64(x) * r64[:, None]
        off_xhat, source = ref.U32 * np.abs(xhat), dict(x=x.cuda())
    got = taco.rmsnorm_backward(dy.cuda(), rstd.cuda(), cuda(w), dsummed=cuda(ds), block=block or 128, code=code, **source)
    dx, dw, off_dx, off_dw = gr.rmsnorm_grads(ref.f64(dy), xhat, r64, ref.f64(w) if affine else None, off_xhat)
    if dsummed:
        dx = dx + ref.f64(ds)
        off_dx = off_dx + 2 * ref.U32 * (np.abs(dx) + np.abs(ref.f64(ds)))
    ref.within(got.dx, dx, off_dx, what="dx")
    assert (got.dweight is None) == (w is None)
    if affine:
        ref.within(got.dweight, dw, off_dw, what="dweight")
    return got


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF16, F32), (F16, F16), (F32, F32), (BF16, BF16)])
def test_grad(taco, rows, hidden, dtype, pdtype):
    check_grad(taco, rows, hidden, dtype, pdtype)
    check_grad(taco, rows, hidden, dtype, pdtype, dsummed=True)
    check_grad(taco, rows, hidden, dtype, pdtype, affine=False)


@pytest.mark.parametrize("block", (32, 64, 128, 256, 512))
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_grad_from_records(taco, block, code, dtype):
    for rows, hidden in ((1, block), (5, 3 * block), (3, 2560), (2, 9216), (2, 34816), (340, 512)):
        if hidden % block == 0:
            check_grad(taco, rows, hidden, dtype, F32, block=block, code=code, dsummed=rows != 5)


def test_grad_from_forward_and_differences(taco):
    """dx and dweight of a scalar loss against central differences of the norm in 64 bits."""
    rows, hidden = 5, 96
    x, r = values(1, rows, hidden), values(2, rows, hidden)
    w, dy, ds = 1 + 0.3 * values(3, hidden), values(4, rows, hidden), values(5, rows, hidden)
    n = taco.rmsnorm(x.cuda(), w.cuda(), eps=EPS, residual=r.cuda())
    g = taco.rmsnorm_backward(dy.cuda(), n.rstd, w.cuda(), x=n.summed, dsummed=ds.cuda())
    h0, w0, dy0, ds0 = ref.f64(n.summed), ref.f64(w), ref.f64(dy), ref.f64(ds)
    loss = lambda h, wt: (gr.rmsnorm(h, wt, EPS)[0] * dy0).sum() + (h * ds0).sum()
    rng = np.random.default_rng(0)
    for _ in range(4):
        along, wl = rng.standard_normal((rows, hidden)), rng.standard_normal(hidden)
        # central differences: 1e-10 of the curvature, 1e-11 of 64-bit rounding over h; the gradient itself 32-bit
        scale = np.abs(ref.f64(g.dx) * along).sum()
        assert abs((ref.f64(g.dx) * along).sum() - gr.difference(lambda h: np.array(loss(h, w0)), h0, along)) <= 1e-5 * scale
        scale = np.abs(ref.f64(g.dweight) * wl).sum()
        assert abs((ref.f64(g.dweight) * wl).sum() - gr.difference(lambda v: np.array(loss(h0, v)), w0, wl)) <= 1e-5 * scale


def test_compressed_records_are_read(taco):
    """Records of compress(variant="ds_only"), whose scales are no powers of two."""
    rows, hidden = 12, 1024
    xhat = values(3, rows, hidden).to(BF16)
    packed = taco.compress(xhat.cuda(), 128, variant="ds_only")
    q, alpha, s = ref.split(packed, 128)
    v = (ref.code_values("e4m3")[q] * s[:, None]).reshape(rows, hidden)
    dy, rstd = values(4, rows, hidden).to(BF16), torch.ones(rows)
    got = taco.rmsnorm_backward(dy.cuda(), rstd.cuda(), torch.ones(hidden).cuda(), packed=packed)
    dx, dw, off_dx, off_dw = gr.rmsnorm_grads(ref.f64(dy), v, ref.f64(rstd), None, 2 * ref.U32 * np.abs(v))
    ref.within(got.dx, dx, off_dx)
    ref.within(got.dweight, dw, off_dw)


def test_repeats_streams_and_graphs(taco):
    """The same bits from run to run, on another stream and from a replayed graph."""
    x, r, dy = (values(i, 700, 1111).to(BF16).cuda() for i in range(3))
    w = (1 + 0.1 * values(7, 1111)).cuda()

    def step():
        n = taco.rmsnorm(x, w, residual=r)
        g = taco.rmsnorm_backward(dy, n.rstd, w, x=n.summed, dsummed=dy)
        return n.y, n.rstd, n.summed, g.dx, g.dweight

    first = [t.clone() for t in step()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = taco.rmsnorm(x, w, residual=r, stream=side).y
    side.synchronize()
    assert torch.equal(y, first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(values(20, 700, 1111).to(BF16))
    want = [t.clone() for t in step()]
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("rows,hidden", [(3, 1001), (153, 1111), (306, 640), (2, 20481), (5, 13)])
def test_nothing_behind_the_tensors(taco, rows, hidden, dtype):
    """What lies in front of and behind the outputs stays as it was, and what lies behind the inputs (NaN) is not read."""
    from fp8_compression_tensor_gb300 import _gated
    lib, stream, n = _gated._library(), torch.cuda.current_stream().cuda_stream, rows * hidden
    pad = 64
    nan = float("nan")
    fill = lambda t: torch.cat([t.reshape(-1).to(dtype), torch.full((pad,), nan, dtype=dtype)]).cuda()
    x, r, dy, ds = (fill(values(i, rows, hidden)) for i in range(4))
    w = torch.cat([1 + 0.1 * values(8, hidden), torch.full((pad,), nan)]).cuda()
    y, s, dx = (torch.full((n + pad,), 7.0, dtype=dtype, device="cuda") for _ in range(3))
    rstd, dw = torch.full((rows + pad,), 7.0, device="cuda"), torch.full((hidden + pad,), 7.0, device="cuda")
    kind = taco._training.DTYPES[dtype]
    a = _gated._RmsNormArgs(x=x.data_ptr(), residual=r.data_ptr(), weight=w.data_ptr(), y=y.data_ptr(), summed=s.data_ptr(),
                            rstd=rstd.data_ptr(), rows=rows, hidden=hidden, eps=EPS, dtype=kind, param_dtype=2)
    assert lib.taco_rmsnorm(ctypes.byref(a), stream) == 0
    need = lib.taco_rmsnorm_backward_workspace(rows, hidden)
    ws = torch.full((need + pad,), 7, dtype=torch.uint8, device="cuda")
    b = _gated._RmsNormBackwardArgs(dy=dy.data_ptr(), x=s.data_ptr(), rstd=rstd.data_ptr(), weight=w.data_ptr(),
                                    dsummed=ds.data_ptr(), dx=dx.data_ptr(), dweight=dw.data_ptr(), workspace=ws.data_ptr(),
                                    workspace_bytes=need, rows=rows, hidden=hidden, dtype=kind, param_dtype=2)
    assert lib.taco_rmsnorm_backward(ctypes.byref(b), stream) == 0
    torch.cuda.synchronize()
    for t, k in ((y, n), (s, n), (dx, n), (rstd, rows), (dw, hidden)):
        assert torch.all(t[k:] == 7) and not torch.isnan(t[:k]).any()
    assert torch.all(ws[need:] == 7)
    want = taco.rmsnorm(x[:n].view(rows, hidden).clone(), w[:hidden].clone(), eps=EPS, residual=r[:n].view(rows, hidden).clone())
    assert torch.equal(want.y.reshape(-1), y[:n])
