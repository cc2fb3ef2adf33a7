"""examples/mlp_block_8bit.py: the training operators together, against the
same block in 64 bits.

What separates the two is the rounding of the bf16 tensors (unit roundoff 2^-8)
and of the records.  E4M3 values are within 2^-4 of the true ones (half of a
step of 1/8), INT8 values within 2^-7 of a block's maximum (the scale's power of
two costs up to a factor of two of 1/254).  An average over many elements
of such errors, uniform within the bound, has a relative root mean square below
2^-4 / sqrt 3 = 0.036 for E4M3; the gradients pass two records (xhat and u), so
their relative error in the 2-norm stays below 0.1.  The output passes none: a few bf16 roundings, below 2^-6.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mlp_block_8bit", os.path.join(ROOT, "examples", "mlp_block_8bit.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(x, residual, gamma, beta, w1, b1, w2, b2):
    h = x + residual
    n = torch.nn.functional.layer_norm(h, h.shape[-1:], gamma, beta)
    return torch.nn.functional.gelu(n @ w1.t() + b1) @ w2.t() + b2 + h


@pytest.mark.parametrize("code,block,tokens,hidden", [("e4m3", 128, 300, 512), ("int8", 64, 77, 256), ("e4m3", 512, 1030, 1024)])
def test_against_64_bits(example, code, block, tokens, hidden):
    params = example.parameters(hidden, 4 * hidden)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, residual, dout = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    args = [x.requires_grad_(), residual.requires_grad_(), *params]
    out = example.mlp_block(*args, block=block, code=code)
    grads = torch.autograd.grad(out, args, dout)
    exact = [a.detach().double().requires_grad_() for a in args]
    want = plain(*exact)
    wanted = torch.autograd.grad(want, exact, dout.double())
    far = lambda a, b: float((a.detach().double() - b.detach()).norm() / b.detach().norm())
    assert far(out, want) < 2.0 ** -6
    for name, a, b in zip(("x", "residual", "gamma", "beta", "w1", "b1", "w2", "b2"), grads, wanted):
        assert a.dtype == args[("x", "residual", "gamma", "beta", "w1", "b1", "w2", "b2").index(name)].dtype
        assert far(a, b) < 0.1, (name, far(a, b))


def test_trains(example, capsys):
    example.main(tokens=512, hidden=256, steps=12)
    lines = [line for line in capsys.readouterr().out.splitlines() if line.startswith("step")]
    assert float(lines[-1].split()[-1]) < 0.9 * float(lines[0].split()[-1])
