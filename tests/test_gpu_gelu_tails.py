"""GELU where it is small: its value and slope below zero, to a few roundings
of their own size.

Bounds, with U = 2^-24, for u < 0 and a = |u|.  erf form: the exponent -a^2/2
log2(e) carries three roundings, which weigh a^2/2 each, and the exponential 4 U
more; the tail q = E t Q(t) adds 3 U of the fit, 3 U of its evaluation, 11 U
through t = 1 / (1 + 0.3 a) and 2 U of products; a phi(a) and the difference a
few more: (1.5 a^2 + 32) U of Phi(u) + a phi(a), and nothing below 2^-120 counts
(E vanishes below 2^-126, a factor of at most 32 before it).  tanh form: exp(-2
v) with six roundings in its exponent 2 |v|, then the reciprocal, the products:
(12 |v| + 16) U of the terms' sizes, and nothing below 2^-116.
"""
import math

import numpy as np
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = ref.U32


@pytest.fixture(scope="module")
def taco():
    import fp8_compression_tensor_gb300 as t
    return t


def gelu_below_zero(u, tanh):
    """gelu(u), its slope, and the bounds on both, for u < 0 in 64 bits."""
    a = np.abs(u)
    if tanh:
        v = math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)
        e = np.exp(2 * v)
        p, rest = e / (1 + e), e / (1 + e) ** 2
        bend = 2 * u * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u ** 2) * rest
        count, least = 12 * np.abs(v) + 16, 2.0 ** -116
    else:
        p = ref.gelu(u, False)[0] / u
        bend = u * np.exp(-u * u / 2) / math.sqrt(2 * math.pi)
        count, least = 1.5 * a ** 2 + 32, 2.0 ** -120
    return u * p, p + bend, count * U * a * p + least, count * U * (p + np.abs(bend)) + least


def records_below_zero(seed, rows, hidden, block):
    """INT8 records of values in (-13, 0) on a grid of its own for every block, and the values."""
    rng = np.random.default_rng(seed)
    q = rng.integers(-127, 0, (rows * hidden // block, block)).astype(np.int8)
    s = (13 / 127 * rng.uniform(0.05, 1.0, (len(q), 1))).astype("<f4")
    tail = np.concatenate([np.ones_like(s), s], 1).view(np.uint8)
    packed = torch.from_numpy(np.concatenate([q.view(np.uint8), tail], 1).reshape(-1).copy())
    return packed, (q.astype(np.float32) * s).astype(np.float64).reshape(rows, hidden)


@pytest.mark.parametrize("tanh", (False, True))
@pytest.mark.parametrize("dtype", (F32, BF16, F16))
def test_gradient_below_zero(taco, tanh, dtype):
    packed, u = records_below_zero(1, 300, 512, 32)
    y, slope, off_y, off_slope = gelu_below_zero(u, tanh)
    dy = torch.randn(300, 512, generator=torch.Generator().manual_seed(2)).to(dtype)
    g = taco.gelu_backward(dy.cuda(), packed.cuda(), approximate="tanh" if tanh else "none", recompute=True, block=32, code="int8")
    d = ref.f64(dy)
    ref.within(g.dx, d * slope, np.abs(d) * (off_slope + U * np.abs(slope)), what="dx")
    ref.within(g.y, y, off_y, what="y again")


@pytest.mark.parametrize("tanh", (False, True))
@pytest.mark.parametrize("hidden", (512, 515))
def test_value_below_zero(taco, tanh, hidden):
    x = -13 * torch.rand(64, hidden, generator=torch.Generator().manual_seed(3)) - 1e-3
    y, _, off, _ = gelu_below_zero(ref.f64(x), tanh)
    ref.within(taco.gelu(x.cuda(), approximate="tanh" if tanh else "none", checkpoint=False).y, y, off, what="y")
