"""Plain implementations of the RMS norm and the gated linear layer in 64 bits
(NumPy) and the error bounds of the kernels' 32-bit arithmetic, in the terms of
training_reference.py (u = 2^-24, sums of `depth(width)` additions one after
another at most)."""
import math

import numpy as np

from training_reference import U32, depth, gelu, slope_bound


def rmsnorm(h: np.ndarray, weight, eps: float):
    """y, rstd, xhat, and the bounds on rstd and xhat."""
    rstd = 1 / np.sqrt((h ** 2).mean(1) + eps)
    xhat = h * rstd[:, None]
    # rstd: half of the mean square's relative error, then the root and its correction
    off_rstd = rstd * (depth(h.shape[1]) / 2 + 8) * U32
    off_xhat = np.abs(h) * off_rstd[:, None] + 2 * U32 * np.abs(xhat)
    return xhat * (1 if weight is None else weight), rstd, xhat, off_rstd, off_xhat


def rmsnorm_grads(dy, xhat, rstd, weight, off_xhat=0.0):
    """dx, dweight and the bounds on their 32-bit errors."""
    a = dy * (1 if weight is None else weight)
    ax, r = a * xhat, rstd[:, None]
    c = ax.mean(1, keepdims=True)
    off_c = (depth(dy.shape[1]) + 4) * U32 * np.abs(ax).mean(1, keepdims=True) + (np.abs(a) * off_xhat).mean(1, keepdims=True)
    off_dx = r * (np.abs(xhat) * off_c + np.abs(c) * off_xhat + 8 * U32 * (np.abs(a) + np.abs(xhat * c)))
    off_dw = (dy.shape[0] + 16) * U32 * np.abs(dy * xhat).sum(0) + (np.abs(dy) * off_xhat).sum(0)
    return r * (a - xhat * c), (dy * xhat).sum(0), off_dx, off_dw


def product(a: np.ndarray, b: np.ndarray):
    """a b^T and the bound on a tensor core's sums: each of K exact products, and
    the accumulator that they join, is cut to 24 bits of the largest addend."""
    return a @ b.T, (a.shape[1] + 64) * U32 * (np.abs(a) @ np.abs(b).T)


def activation(g: np.ndarray, name: str):
    """act(g) and its slope."""
    if name == "silu":
        with np.errstate(over="ignore"):
            p = 1 / (1 + np.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    return gelu(g, name == "gelu_tanh")


STEEPEST = 1.13   # largest slope of the three activations


def value_bound(g: np.ndarray) -> np.ndarray:
    """32-bit error of act(g): the gate in [0, 1] to eight roundings, times g."""
    return 8 * U32 * np.abs(g)


def gated(z: np.ndarray, off_z, name: str):
    """y = act(z_gate) z_up and its bound."""
    inner = z.shape[1] // 2
    g, u = z[:, :inner], z[:, inner:]
    off_g, off_u = (off_z[:, :inner], off_z[:, inner:]) if isinstance(off_z, np.ndarray) else (off_z, off_z)
    value = activation(g, name)[0]
    off_value = STEEPEST * off_g + value_bound(np.abs(g) + off_g)
    return value * u, off_value * (np.abs(u) + off_u) + np.abs(value) * off_u + 2 * U32 * np.abs(value * u)


def gated_grads(dy: np.ndarray, z: np.ndarray, name: str):
    """dz and its bound."""
    inner = z.shape[1] // 2
    g, u = z[:, :inner], z[:, inner:]
    value, slope = activation(g, name)
    dz = np.concatenate([dy * u * slope, dy * value], 1)
    off = np.concatenate([np.abs(dy * u) * slope_bound(g), np.abs(dy) * value_bound(g)], 1)
    return dz, off + 4 * U32 * np.abs(dz)


def column_sums(dz: np.ndarray, off: np.ndarray):
    """Sums over rows of 32-bit values that are off by `off` each."""
    return dz.sum(0), (dz.shape[0] + 16) * U32 * np.abs(dz).sum(0) + off.sum(0)


def difference(f, at: np.ndarray, along: np.ndarray, h: float = 1e-5) -> float:
    """The slope of f at `at` along a direction, by central differences."""
    return float(math.fsum(((f(at + h * along) - f(at - h * along)) / (2 * h)).reshape(-1)))
