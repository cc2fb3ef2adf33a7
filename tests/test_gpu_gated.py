"""The gated linear layer and its gradient against plain implementations in 64
bits, at the sizes, types and values where they can go wrong.  The bounds are
those of gated_reference.py."""
import ctypes

import numpy as np
import pytest
import torch

import gated_reference as gr
import training_reference as ref
from test_gpu_rmsnorm import check_records, cuda, values

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CODES = ("e4m3", "e5m2", "int8")
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    yield t
    assert t.device_status() == 0


def check_forward(taco, rows, hidden, inner, dtype=BF16, activation="silu", bias=None, block=None, code="e4m3"):
    x = values(rows + hidden, rows, hidden).to(dtype)
    w = (values(inner, 2 * inner, hidden) * hidden ** -0.5).to(dtype)
    b = (0.3 * values(5, 2 * inner)).to(bias) if bias else None
    got = taco.gated_linear(x.cuda(), w.cuda(), cuda(b), activation=activation, checkpoint=block is not None,
                            block=block or 128, code=code)
    z, off_z = gr.product(ref.f64(x), ref.f64(w))
    if bias:
        z = z + ref.f64(b)
        off_z = off_z + ref.U32 * np.abs(z)
    y, off_y = gr.gated(z, off_z, activation)
    assert got.y.shape == (rows, inner) and got.y.dtype == dtype
    ref.within(got.y, y, off_y, what="y")
    if block:
        check_records(got.packed, z, off_z, rows, 2 * inner, block, code)
    return got


# One of everything, odd sizes, the neighbours of tiles of 16, 64, 128 and 256, few rows (the serving form) and more tiles than SMs.
SHAPES = [(1, 1, 1), (3, 7, 5), (1, 64, 32), (5, 8, 33), (130, 72, 100), (257, 1000, 160), (128, 512, 256), (300, 520, 300),
          (16, 2048, 384), (17, 1111, 65), (1, 4096, 1000), (64, 264, 4096), (65, 64, 130), (33, 63, 64), (255, 128, 127),
          (513, 96, 1000), (1000, 40, 2500), (2, 8200, 72), (9, 136, 20000), (1100, 200, 24)]


@pytest.mark.parametrize("rows,hidden,inner", SHAPES)
@pytest.mark.parametrize("dtype", (BF16, F16))
def test_forward(taco, rows, hidden, inner, dtype):
    check_forward(taco, rows, hidden, inner, dtype)
    check_forward(taco, rows, hidden, inner, dtype, "gelu", bias=F32 if rows % 2 else dtype)


@pytest.mark.parametrize("rows", (1, 2, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 192, 256, 320))
def test_forward_every_row_count(taco, rows):
    """Both sides of every limit on the number of rows."""
    check_forward(taco, rows, 320, 200)
    check_forward(taco, rows, 1096, 72, F16, "gelu_tanh", bias=BF16)


@pytest.mark.parametrize("activation", ACTIVATIONS)
@pytest.mark.parametrize("block", (32, 64, 128))
@pytest.mark.parametrize("code", CODES)
def test_forward_records(taco, activation, block, code):
    for rows, hidden, inner in ((1, 72, block), (37, 256, 5 * block), (260, 100, 384), (129, 33, 2 * block)):
        for dtype, bias in ((BF16, None), (F16, F32)):
            check_forward(taco, rows, hidden, inner, dtype, activation, bias, block, code)


def test_forward_keeps_with_and_without_records(taco):
    """The same y with a checkpoint and without one, above the serving form's rows."""
    x, w = values(1, 300, 256).to(BF16).cuda(), (values(2, 512, 256) / 16).to(BF16).cuda()
    assert torch.equal(taco.gated_linear(x, w).y, taco.gated_linear(x, w, checkpoint=True).y)


def test_forward_leading_dimensions_and_empty(taco):
    x, w = values(1, 2, 3, 64).to(BF16).cuda(), values(2, 40, 64).to(BF16).cuda()
    y = taco.gated_linear(x, w).y
    assert y.shape == (2, 3, 20) and torch.equal(y.view(6, 20), taco.gated_linear(x.view(6, 64), w).y)
    assert taco.gated_linear(x[:0].contiguous(), w).y.shape == (0, 3, 20)
    assert taco.gated_linear(x, w[:0].contiguous()).y.shape == (2, 3, 0)
    with pytest.raises(ValueError):
        taco.gated_linear(x, w[:39].contiguous())
    with pytest.raises(ValueError):
        taco.gated_linear(x.transpose(0, 1), w)
    with pytest.raises(TypeError):
        taco.gated_linear(x.float(), w.float())
    with pytest.raises(TypeError):
        taco.gated_linear(x, w.half())
    with pytest.raises(taco.TacoError):
        taco.gated_linear(x, values(2, 512, 64).to(BF16).cuda(), checkpoint=True, block=256)


@pytest.mark.parametrize("rows", (4, 300))
def test_forward_non_finite(taco, rows):
    """A NaN or an infinity in x spoils its own row only, in W its own column only."""
    x, w = values(1, rows, 200).to(BF16).cuda(), (values(2, 256, 200) / 14).to(BF16).cuda()
    clean = taco.gated_linear(x, w, checkpoint=rows > 256)
    for bad in (float("nan"), float("inf")):
        xb, wb = x.clone(), w.clone()
        xb[2, 199] = bad
        got = taco.gated_linear(xb, w, checkpoint=rows > 256)
        keep = torch.arange(rows, device="cuda") != 2
        assert torch.equal(got.y[keep], clean.y[keep]) and not torch.isfinite(got.y[2]).all()
        if got.packed is not None:
            v = taco.decompress(got.packed, rows, 256, variant="ds_only")
            assert torch.isnan(v[2]).all() and torch.isfinite(v[keep]).all()
        wb[70, 0] = bad
        got = taco.gated_linear(x, wb)
        keep = torch.arange(128, device="cuda") != 70
        assert torch.equal(got.y[:, keep], clean.y[:, keep]) and not torch.isfinite(got.y[:, 70]).any()


def test_forward_large_values(taco):
    """Gates far out on both sides: silu and gelu vanish below and are the identity above."""
    x = torch.tensor([[1.0]], dtype=BF16).cuda()
    gates = torch.tensor([-3e38, -1e30, -200.0, -90.0, 0.0, 90.0, 200.0, 1e30], dtype=BF16)
    for name in ACTIVATIONS:
        y = taco.gated_linear(x, torch.cat([gates, torch.ones_like(gates)])[:, None].contiguous().cuda(), activation=name).y[0].cpu()
        assert torch.all(y[:5].float().abs() < 1e-30) and torch.equal(y[5:], gates[5:])


def check_backward(taco, rows, hidden, inner, dtype=BF16, activation="silu", bias=None, block=32, code="e4m3", again=False):
    z = values(rows + inner, rows, 2 * inner, scale=1.5)
    packed = ref.make_records(z, block, code)
    z = ref.decode(packed, rows, 2 * inner, block, code)
    dy = values(3, rows, inner, scale=0.1).to(dtype)
    w = (values(4, 2 * inner, hidden) * hidden ** -0.5).to(dtype) if hidden else None
    got = taco.gated_linear_backward(dy.cuda(), packed.cuda(), cuda(w), activation=activation, bias_dtype=bias,
                                     recompute=again, block=block, code=code)
    dz, off = gr.gated_grads(ref.f64(dy), z, activation)
    ref.within(got.dz, dz, off, what="dz")
    if hidden:
        # the product of dz as it is written
        dx, off_dx = gr.product(ref.f64(got.dz), ref.f64(w).T.copy())
        ref.within(got.dx, dx, off_dx, what="dx")
    if bias:
        ref.within(got.dbias, *gr.column_sums(dz, off), what="dbias")
    if again:
        ref.within(got.y, *gr.gated(z, 0.0, activation), what="y")
    assert (got.dx is None, got.dbias is None, got.y is None) == (not hidden, bias is None, not again)
    return got


@pytest.mark.parametrize("rows,hidden,inner", [(1, 1, 32), (3, 7, 64), (130, 72, 128), (257, 1000, 160), (300, 521, 320),
                                               (16, 2048, 384), (17, 1111, 96), (1, 4096, 1024), (513, 96, 1024), (2, 8200, 96),
                                               (9, 0, 20000), (1100, 200, 32), (700, 264, 2560), (255, 256, 256)])
@pytest.mark.parametrize("dtype", (BF16, F16))
def test_backward(taco, rows, hidden, inner, dtype):
    check_backward(taco, rows, hidden, inner, dtype)
    check_backward(taco, rows, hidden, inner, dtype, "gelu", bias=F32, again=True)


@pytest.mark.parametrize("activation", ACTIVATIONS)
@pytest.mark.parametrize("block", (32, 64, 128))
@pytest.mark.parametrize("code", CODES)
def test_backward_records(taco, activation, block, code):
    for rows, hidden, inner, dtype in ((1, 8, block, BF16), (37, 40, 5 * block, F16), (600, 0, 3 * block, BF16)):
        check_backward(taco, rows, hidden, inner, dtype, activation, dtype, block, code, again=True)


def test_backward_empty(taco):
    dy = torch.empty(0, 256, device="cuda", dtype=BF16)
    w = values(1, 512, 64).to(BF16).cuda()
    g = taco.gated_linear_backward(dy, torch.empty(0, dtype=torch.uint8, device="cuda"), w, bias_dtype=F32, recompute=True)
    assert g.dz.shape == (0, 512) and g.dx.shape == (0, 64) and g.y.shape == (0, 256) and not g.dbias.any()
    with pytest.raises(ValueError):
        taco.gated_linear_backward(dy[:, :0].contiguous(), torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        taco.gated_linear_backward(dy, torch.empty(0, dtype=torch.uint8, device="cuda"), w[:, :0].contiguous())


@pytest.mark.parametrize("activation", ACTIVATIONS)
def test_backward_differences(taco, activation):
    """dz against central differences of the layer's product in 64 bits."""
    rows, inner = 6, 96
    packed = ref.make_records(values(1, rows, 2 * inner, scale=2.0), 32, "int8")
    z, dy = ref.decode(packed, rows, 2 * inner, 32, "int8"), values(2, rows, inner).to(F16)
    got = taco.gated_linear_backward(dy.cuda(), packed.cuda(), activation=activation, block=32, code="int8")
    loss = lambda v: np.array((gr.gated(v, 0.0, activation)[0] * ref.f64(dy)).sum())
    rng = np.random.default_rng(1)
    dz, off = gr.gated_grads(ref.f64(dy), z, activation)
    off = off + ref.UNIT[F16] * np.abs(dz) + ref.TINY[F16]
    for _ in range(4):
        along = rng.standard_normal(z.shape)
        slack = (off * np.abs(along)).sum() + 1e-7 * np.abs(dz * along).sum()
        assert abs((ref.f64(got.dz) * along).sum() - gr.difference(loss, z, along)) <= slack


def test_backward_from_forward_and_weight_gradient(taco):
    """Forward, backward and weight_grad on each other's buffers."""
    rows, hidden, inner = 300, 256, 384
    x, w = values(1, rows, hidden).to(BF16), (values(2, 2 * inner, hidden) / 16).to(BF16)
    dy = values(3, rows, inner, scale=0.1).to(BF16)
    n = taco.rmsnorm(x.cuda(), checkpoint=True)
    f = taco.gated_linear(n.y, w.cuda(), checkpoint=True)
    g = taco.gated_linear_backward(dy.cuda(), f.packed, w.cuda(), recompute=True)
    z = ref.decode(f.packed, rows, 2 * inner, 128, "e4m3")
    ref.within(g.dz, *gr.gated_grads(ref.f64(dy), z, "silu"))
    ref.within(g.y, *gr.gated(z, 0.0, "silu"))
    dw = taco.weight_grad(g.dz, n.packed, hidden)
    want, off = gr.product(ref.f64(g.dz).T.copy(), ref.decode(n.packed, rows, hidden, 128, "e4m3").T.copy())
    ref.within(dw, want, off)


def test_repeats_streams_and_graphs(taco):
    """The same bits from run to run, on other streams at once and from replayed graphs."""
    shapes = [(5, 1024, 640), (300, 264, 512), (40, 333, 256)]
    made = []
    for rows, hidden, inner in shapes:
        x, w = values(1, rows, hidden).to(BF16).cuda(), (values(2, 2 * inner, hidden) / 16).to(BF16).cuda()
        b, dy = values(4, 2 * inner).cuda(), values(3, rows, inner).to(BF16).cuda()

        def step(x=x, w=w, b=b, dy=dy):
            serve = taco.gated_linear(x, w, b)
            f = taco.gated_linear(x, w, b, checkpoint=True)
            g = taco.gated_linear_backward(dy, f.packed, w, bias_dtype=F32, recompute=True)
            return serve.y, f.y, f.packed, g.dz, g.dx, g.dbias, g.y

        made.append((x, step))
    first = [[t.clone() for t in step()] for _, step in made]
    for (_, step), want in zip(made, first):
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(want, step()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    outs = []
    for (_, step), s in zip(made, streams):
        with torch.cuda.stream(s):
            outs.append([step() for _ in range(5)])
    torch.cuda.synchronize()
    for got, want in zip(outs, first):
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(want, one))
    graphs = []
    for x, step in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for (x, step), (g, out) in zip(made, graphs):
        x.copy_(values(9, *x.shape).to(BF16))
        want = [t.clone() for t in step()]
        for t in out:
            t.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("rows,hidden,inner,block", [(1, 72, 96, 32), (3, 33, 37, None), (130, 136, 160, 32), (257, 64, 384, 128),
                                                     (40, 200, 136, None), (300, 50, 77, None), (129, 1024, 64, 64)])
def test_nothing_behind_the_tensors(taco, rows, hidden, inner, block):
    """What lies behind the outputs stays as it was, and what lies behind the inputs (NaN) is not read."""
    from fp8_compression_tensor_gb300 import _gated
    lib, stream, pad = _gated._library(), torch.cuda.current_stream().cuda_stream, 4096
    nan = lambda t: torch.cat([t.reshape(-1), torch.full((pad,), float("nan"), dtype=t.dtype)]).cuda()
    x, w = values(1, rows, hidden).to(BF16), (values(2, 2 * inner, hidden) / hidden ** 0.5).to(BF16)
    dy = values(3, rows, inner).to(BF16)
    px, pw, pdy = nan(x), nan(w), nan(dy)
    out = lambda n, t=BF16: torch.full((n + pad,), 7, dtype=t, device="cuda")
    y, dz, dx, again = out(rows * inner), out(2 * rows * inner), out(rows * hidden), out(rows * inner)
    nbytes = taco.compressed_bytes(rows, 2 * inner, block) if block else 0
    packed, dbias = out(nbytes, torch.uint8), out(2 * inner, F32)
    need = lib.taco_gated_linear_workspace(rows, inner, hidden)
    ws = out(need, torch.uint8)
    a = _gated._GatedLinearArgs(x=px.data_ptr(), weight=pw.data_ptr(), y=y.data_ptr(), packed=packed.data_ptr() if block else 0,
                                workspace=ws.data_ptr(), workspace_bytes=need, rows=rows, inner=inner, hidden=hidden,
                                param_dtype=2, block=block or 0)
    assert lib.taco_gated_linear(ctypes.byref(a), stream) == 0
    torch.cuda.synchronize()
    assert torch.all(y[rows * inner:] == 7) and torch.all(packed[nbytes:] == 7) and torch.all(ws[need:] == 7)
    want = taco.gated_linear(x.cuda(), w.cuda(), checkpoint=block is not None, block=block or 128)
    assert torch.equal(want.y.reshape(-1), y[:rows * inner]) and torch.isfinite(want.y).all()
    if not block:
        return
    assert torch.equal(want.packed, packed[:nbytes])
    need = lib.taco_gated_linear_backward_workspace(rows, inner, hidden)
    ws = out(need, torch.uint8)
    b = _gated._GatedLinearBackwardArgs(dy=pdy.data_ptr(), packed=packed.data_ptr(), weight=pw.data_ptr(), dz=dz.data_ptr(),
                                        dx=dx.data_ptr(), y=again.data_ptr(), dbias=dbias.data_ptr(), workspace=ws.data_ptr(),
                                        workspace_bytes=need, rows=rows, inner=inner, hidden=hidden, param_dtype=2, block=block)
    assert lib.taco_gated_linear_backward(ctypes.byref(b), stream) == 0
    torch.cuda.synchronize()
    for t, n in ((dz, 2 * rows * inner), (dx, rows * hidden), (again, rows * inner), (dbias, 2 * inner), (ws, need)):
        assert torch.all(t[n:] == 7)
    g = taco.gated_linear_backward(dy.cuda(), want.packed, w.cuda(), bias_dtype=F32, recompute=True, block=block)
    assert torch.equal(g.dx.reshape(-1), dx[:rows * hidden]) and torch.isfinite(g.dx).all()
    assert torch.equal(g.dbias, dbias[:2 * inner])
