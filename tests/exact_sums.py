"""Inputs whose products sum to whole numbers below 2^24 in every partial sum, so
that binary32 sums are exact in any order, and what the gated layer and its
gradient make of them: a term that is lost, taken twice or taken from elsewhere
shows in the outputs, however long the sum.

The layer: x and W hold -1, 0 and 1, W's up rows 1 / 32 of that (f16 then holds
y); the gate's bias is 1024 and the sums stay within 1000, so the gate's sigmoid is
1 in binary32 (exp(-24) < 2^-25) and 32 y the product of two whole numbers below
2^11, rounded once.  The gradient: z_gate = 32,
where SiLU is 32 and its slope 1, z_up and dy are -1, 0 and 1."""
import torch

GATE = 1024.0


def signs(seed, *shape, density=1.0, device="cpu"):
    """-1 and 1 with this density, 0 elsewhere."""
    g = torch.Generator(device=device).manual_seed(seed)
    t = torch.randint(0, 2, shape, generator=g, device=device, dtype=torch.int8).mul_(2).sub_(1)
    if density < 1:
        t *= torch.rand(shape, generator=g, device=device) < density
    return t


def layer(rows, hidden, inner, seed=0, device="cpu"):
    """x, W and the bias: sums of about 15000 terms at most, 120 large (a thousand is eight times that)."""
    x, w = signs(seed, rows, hidden, device=device), signs(seed + 1, 2 * inner, hidden, density=min(2 / 3, 15000 / hidden), device=device)
    w = w.to(torch.bfloat16)
    w[inner:] /= 32
    bias = torch.zeros(2 * inner, device=device)
    bias[:inner] = GATE
    return x, w, bias


def layer_values(x, w, bias):
    """z, whole numbers, and y before its rounding."""
    z = x.float() @ w.float().t()
    assert float(z.abs().max()) < 1000
    z += bias
    inner = w.shape[0] // 2
    return z, z[:, :inner] * z[:, inner:]


def gradient(rows, hidden, inner, seed=0, device="cpu"):
    """dy, z_up and W."""
    return (signs(seed, rows, inner, density=2 / 3, device=device), signs(seed + 1, rows, inner, density=2 / 3, device=device),
            signs(seed + 2, 2 * inner, hidden, density=2 / 3, device=device))


def gradient_values(dy, up, w):
    """dz, dx and dbias before their roundings."""
    dz = torch.cat([dy * up, 32 * dy], 1).float()
    assert 32 * 2 * up.shape[1] < 2 ** 24 and 32 * dy.shape[0] < 2 ** 24
    return dz, dz @ w.float(), dz.sum(0)
