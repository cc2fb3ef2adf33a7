"""examples/gated_block_8bit.py: the RMS norm, the gated linear layer, their
gradients and the weight gradient together, against the same block in 64 bits.

What separates the two is the rounding of the bf16 tensors (unit roundoff 2^-8)
and of the records: E4M3 values are within 2^-4 of the true ones, INT8 values
within 2^-7 of a block's maximum, with a relative root mean square below 2^-4 /
sqrt 3 = 0.036 over many elements.  A gradient passes three records (xhat, both
projections), each at most once as a factor and the gate's also through the
activation's slope, so its relative error in the 2-norm stays below 4 times
0.036 = 0.15.  The output passes none: a few bf16 roundings, below 2^-6.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("x", "residual", "gamma", "w", "wd")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_block_8bit", os.path.join(ROOT, "examples", "gated_block_8bit.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(x, residual, gamma, w, wd, activation):
    h = x + residual
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * gamma
    gate, up = (n @ w.t()).chunk(2, -1)
    act = torch.nn.functional.silu(gate) if activation == "silu" else torch.nn.functional.gelu(
        gate, approximate="tanh" if activation == "gelu_tanh" else "none")
    return (act * up) @ wd.t() + h


@pytest.mark.parametrize("activation,code,block,tokens,hidden,inner", [
    ("silu", "e4m3", 128, 300, 512, 1408), ("gelu", "int8", 64, 77, 256, 640), ("gelu_tanh", "e4m3", 32, 1030, 1024, 2720),
    ("silu", "int8", 128, 1, 128, 256)])
def test_against_64_bits(example, activation, code, block, tokens, hidden, inner):
    params = example.parameters(hidden, inner)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, residual, dout = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    args = [x.requires_grad_(), residual.requires_grad_(), *params]
    out = example.gated_block(*args, activation=activation, block=block, code=code)
    grads = torch.autograd.grad(out, args, dout)
    exact = [a.detach().double().requires_grad_() for a in args]
    want = plain(*exact, activation)
    wanted = torch.autograd.grad(want, exact, dout.double())
    far = lambda a, b: float((a.detach().double() - b.detach()).norm() / b.detach().norm())
    assert far(out, want) < 2.0 ** -6
    for name, arg, a, b in zip(NAMES, args, grads, wanted):
        assert a.dtype == arg.dtype and a.shape == arg.shape
        assert far(a, b) < 0.15, (name, far(a, b))


def test_batched_input(example):
    """Leading dimensions are flattened, and a gradient that is not contiguous is taken."""
    params = example.parameters(256, 384)
    x = torch.randn(3, 20, 256, device="cuda").to(torch.bfloat16).requires_grad_()
    out = example.gated_block(x, x.detach(), *params)
    dout = torch.randn(256, 20, 3, device="cuda").to(torch.bfloat16).permute(2, 1, 0)
    grads = torch.autograd.grad(out, [x, *params], dout)
    flat = x.detach().reshape(60, 256).requires_grad_()
    again = torch.autograd.grad(example.gated_block(flat, flat.detach(), *params), [flat, *params], dout.reshape(60, 256))
    assert torch.equal(grads[0].reshape(60, 256), again[0])
    for a, b in zip(grads[1:], again[1:]):
        assert torch.equal(a, b)


def test_runs(example, capsys):
    example.main(tokens=256, hidden=256, inner=640, steps=2)
    assert "kept for the backward pass" in capsys.readouterr().out


def test_second_derivative_is_refused(example):
    params = example.parameters(128, 256)
    x = torch.randn(8, 128, device="cuda").to(torch.bfloat16).requires_grad_()
    dw, = torch.autograd.grad(example.gated_block(x, x.detach(), *params).float().square().sum(), params[1], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dw.float().square().sum().backward()
