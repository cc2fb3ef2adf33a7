"""examples/mlp_block_8bit.py: its gradients come from 8-bit records, outside
autograd, so a derivative of them is refused rather than half of one returned.
The operators are stood in for by plain ones on the CPU."""
import importlib.util
import os
from types import SimpleNamespace

import pytest
import torch

import fp8_compression_tensor_gb300 as taco

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def layernorm(x, weight, bias, residual, checkpoint, block, code):
    h = x + residual
    mean = h.float().mean(-1, keepdim=True)
    rstd = torch.rsqrt((h.float() - mean).square().mean(-1, keepdim=True) + 1e-5)
    xhat = (h.float() - mean) * rstd
    return taco.LayerNorm((xhat * weight + bias).to(x.dtype), mean, rstd, h, xhat)


def layernorm_backward(dy, rstd, weight, packed, dsummed, block, code):
    a = dy.float() * weight
    dx = rstd * (a - a.mean(-1, keepdim=True) - packed * (a * packed).mean(-1, keepdim=True))
    return taco.LayerNormGrads(dx.to(dy.dtype) + dsummed, (dy.float() * packed).sum(0), dy.float().sum(0))


def gelu(x, bias, block, code):
    u = x.float() + bias
    return taco.Gelu(torch.nn.functional.gelu(u).to(x.dtype), u)


def gelu_backward(dy, packed, bias_dtype, recompute, block, code):
    with torch.enable_grad():
        u = packed.detach().requires_grad_()
        y = torch.nn.functional.gelu(u)
        dx, = torch.autograd.grad(y, u, dy.detach().float())
    return taco.GeluGrads(dx.to(dy.dtype), dx.sum(0).to(bias_dtype), y.detach().to(dy.dtype))


def weight_grad(dy, packed, hidden, scale, shift, dy_sum, dtype, block, code):
    return (dy.detach().float().t() @ (packed * scale + shift)).to(dtype).detach()


@pytest.fixture
def example(monkeypatch):
    spec = importlib.util.spec_from_file_location("mlp_block_8bit", os.path.join(ROOT, "examples", "mlp_block_8bit.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.setattr(module, "taco", SimpleNamespace(layernorm=layernorm, layernorm_backward=layernorm_backward, gelu=gelu,
                                                        gelu_backward=gelu_backward, weight_grad=weight_grad))
    return module


def test_second_derivative_is_refused(example):
    params = example.parameters(32, 64, device="cpu")
    x, residual = (torch.randn(8, 32, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).requires_grad_() for i in (1, 2))
    w2 = params[4]
    loss = example.mlp_block(x, residual, *params).float().square().sum()
    dw2, = torch.autograd.grad(loss, w2, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dw2.float().square().sum().backward()
