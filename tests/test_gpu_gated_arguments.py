"""The RMS norm and the gated layer: tensors that do not fit each other are
refused before a launch, and calls from several threads do not disturb each other."""
import threading

import pytest
import torch

from test_gpu_gated import BF16, F16, F32, taco, values  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rmsnorm_arguments(taco):  # noqa: F811
    x, w = values(1, 4, 256).to(BF16).cuda(), torch.ones(256).cuda()
    rstd, packed = torch.ones(4).cuda(), torch.zeros(taco.compressed_bytes(4, 256), dtype=torch.uint8).cuda()
    for error, call in (
            (ValueError, lambda: taco.rmsnorm(x.t())),
            (ValueError, lambda: taco.rmsnorm(x, w[:128].contiguous())),
            (TypeError, lambda: taco.rmsnorm(x, residual=x.float())),
            (ValueError, lambda: taco.rmsnorm(x, residual=x[:2].contiguous())),
            (TypeError, lambda: taco.rmsnorm(x, w.double())),
            (TypeError, lambda: taco.rmsnorm(x.int())),
            (taco.TacoError, lambda: taco.rmsnorm(x, eps=-1.0)),
            (taco.TacoError, lambda: taco.rmsnorm(x, checkpoint=True, block=96)),
            (taco.TacoError, lambda: taco.rmsnorm(x, packed_y=True, block=512)),
            (KeyError, lambda: taco.rmsnorm(x, checkpoint=True, code="e3m4")),
            (ValueError, lambda: taco.rmsnorm_backward(x, rstd, w)),
            (ValueError, lambda: taco.rmsnorm_backward(x, rstd, w, x=x, packed=packed)),
            (ValueError, lambda: taco.rmsnorm_backward(x, rstd[:3].contiguous(), w, x=x)),
            (TypeError, lambda: taco.rmsnorm_backward(x, rstd.half(), w, x=x)),
            (TypeError, lambda: taco.rmsnorm_backward(x, rstd, w, x=x.half())),
            (ValueError, lambda: taco.rmsnorm_backward(x, rstd, w, packed=packed[:-8].contiguous())),
            (ValueError, lambda: taco.rmsnorm_backward(x, rstd, w, x=x, dsummed=x[:1].contiguous()))):
        with pytest.raises(error):
            call()


def test_gated_arguments(taco):  # noqa: F811
    x, w = values(1, 4, 64).to(BF16).cuda(), values(2, 512, 64).to(BF16).cuda()
    dy, packed = values(3, 4, 256).to(BF16).cuda(), torch.zeros(taco.compressed_bytes(4, 512), dtype=torch.uint8).cuda()
    for error, call in (
            (ValueError, lambda: taco.gated_linear(x, w[:, :32].contiguous())),
            (ValueError, lambda: taco.gated_linear(x, w.t())),
            (ValueError, lambda: taco.gated_linear(x, w.view(2, 256, 64))),
            (TypeError, lambda: taco.gated_linear(x, w.half())),
            (TypeError, lambda: taco.gated_linear(x.float(), w.float())),
            (ValueError, lambda: taco.gated_linear(x, w, bias=torch.zeros(256).cuda())),
            (ValueError, lambda: taco.gated_linear(x, w, activation="relu")),
            (taco.TacoError, lambda: taco.gated_linear(x, w, checkpoint=True, block=512)),
            (taco.TacoError, lambda: taco.gated_linear(x, w[:384].contiguous(), checkpoint=True)),
            (ValueError, lambda: taco.gated_linear(x[:, :0].contiguous(), w[:, :0].contiguous())),
            (ValueError, lambda: taco.gated_linear_backward(dy, packed[:-8].contiguous(), w)),
            (TypeError, lambda: taco.gated_linear_backward(dy, packed.float(), w)),
            (TypeError, lambda: taco.gated_linear_backward(dy.float(), packed)),
            (ValueError, lambda: taco.gated_linear_backward(dy, packed, w[:256].contiguous())),
            (TypeError, lambda: taco.gated_linear_backward(dy, packed, w.half())),
            (TypeError, lambda: taco.gated_linear_backward(dy, packed, bias_dtype=torch.float64)),
            (taco.TacoError, lambda: taco.gated_linear_backward(dy, packed[:4 * 2 * 264].contiguous(), block=256))):
        with pytest.raises(error):
            call()


def test_threads(taco):  # noqa: F811
    """Four threads, a stream each, all forms of the calls: the bits of the calls one after another."""
    shapes = [(5, 512, 640, BF16), (300, 264, 512, F16), (130, 333, 256, BF16), (700, 128, 1024, F16)]

    def run(rows, hidden, inner, dtype):
        x, w = values(1, rows, hidden).to(dtype).cuda(), (values(2, 2 * inner, hidden) / 16).to(dtype).cuda()
        n = taco.rmsnorm(x, torch.ones(hidden, device="cuda"), residual=x)
        f = taco.gated_linear(n.y, w, checkpoint=True)
        g = taco.gated_linear_backward(f.y, f.packed, w, bias_dtype=F32, recompute=True)
        d = taco.rmsnorm_backward(g.dx, n.rstd, x=n.summed)
        return taco.gated_linear(n.y, w).y, f.packed, g.dz, g.dbias, g.y, d.dx

    wanted = [run(*s) for s in shapes]
    torch.cuda.synchronize()
    failed = []

    def thread(shape, want):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = run(*shape)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        failed.append(shape)
                    stream.synchronize()
        except Exception as e:   # noqa: BLE001 -- an exception of a thread would be lost
            failed.append(e)

    threads = [threading.Thread(target=thread, args=p) for p in zip(shapes, wanted)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("rows", (40, 300))
def test_padding_rows(taco, rows):  # noqa: F811
    """Rows of zeros (padding) give zeros: all-zero records with s = 0, and no gradient from them."""
    x, w = values(1, rows, 136).to(BF16).cuda(), (values(2, 512, 136) / 12).to(BF16).cuda()
    x[5:17] = 0
    f = taco.gated_linear(x, w, checkpoint=True)
    assert not f.y[5:17].any() and not taco.gated_linear(x, w).y[5:17].any()
    records = f.packed.view(rows, 4, 136)[5:17]
    assert not records[:, :, :128].any() and not records[:, :, 132:].any()
    assert torch.all(records[:, :, 128:132].contiguous().view(torch.float32) == 1)
    g = taco.gated_linear_backward(values(3, rows, 256).to(BF16).cuda(), f.packed, w, recompute=True)
    assert not g.dz[5:17].any() and not g.dx[5:17].any() and not g.y[5:17].any()
    n = taco.rmsnorm(x, checkpoint=False)
    assert not n.y[5:17].any() and torch.isfinite(n.rstd).all()
    assert torch.isfinite(taco.rmsnorm_backward(x, n.rstd, x=x).dx).all()


@pytest.mark.parametrize("rows", (3, 200))
def test_products_beyond_binary32(taco, rows):  # noqa: F811
    """Projections that overflow are infinite: their blocks decode to NaN, other rows and blocks stay."""
    x, w = values(1, rows, 64).to(BF16), values(2, 512, 64).to(BF16)
    clean = taco.gated_linear(x.cuda(), w.cuda(), checkpoint=True)
    x[2] = 1e30
    w[130] = 3e38        # gate column 130: the second block of the gate
    got = taco.gated_linear(x.cuda(), w.cuda(), checkpoint=True)
    v, want = (taco.decompress(r.packed, rows, 512, variant="ds_only") for r in (got, clean))
    assert torch.isnan(v[2, 128:256]).all() and torch.isfinite(v[2, :128]).all() and torch.isfinite(v[2, 256:]).all()
    keep = torch.arange(rows, device="cuda") != 2
    assert torch.equal(v[keep][:, :128], want[keep][:, :128]) and torch.equal(v[keep][:, 256:], want[keep][:, 256:])
