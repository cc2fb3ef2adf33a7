"""Plain implementations of the training operators in 64 bits (NumPy), and the
error bounds that the kernels' 32-bit arithmetic is held to.

u = 2^-24 is binary32's unit roundoff.  A row's sums may be taken in any order
with at most width / 32 + 64 additions one after another (one warp per row is
the least parallel arrangement), so a sum of n terms t is off by at most
depth * u * sum|t|.
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -24
# Unit roundoff of the output types (8, 11 and 24 significant bits).
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
# Absolute rounding error where the type goes subnormal.
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
MANTISSA = {"e4m3": (3, -6), "e5m2": (2, -14)}

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def depth(width: int) -> float:
    return width / 32 + 64


# ---------------------------------------------------------------------------
# Records
# ---------------------------------------------------------------------------

def code_values(code: str) -> np.ndarray:
    """The value of each code byte, from the formats' definitions."""
    out = np.empty(256)
    for b in range(256):
        if code == "int8":
            out[b] = b - 256 if b > 127 else b
            continue
        m_bits, e_min = MANTISSA[code]
        e, m = (b & 127) >> m_bits, b & ((1 << m_bits) - 1)
        v = math.ldexp(m, e_min - m_bits) if e == 0 else math.ldexp(m + (1 << m_bits), e_min + e - 1 - m_bits)
        if code == "e4m3" and b & 127 == 127:
            v = math.nan
        if code == "e5m2" and e == 31:
            v = math.inf if m == 0 else math.nan
        out[b] = -v if b > 127 else v
    return out


def split(packed, block: int):
    rec = packed.cpu().numpy().reshape(-1, block + 8)
    alpha = rec[:, block:block + 4].copy().view("<f4").reshape(-1).astype(np.float64)
    s = rec[:, block + 4:].copy().view("<f4").reshape(-1).astype(np.float64)
    return rec[:, :block], alpha, s


def decode(packed, rows: int, hidden: int, block: int, code: str) -> np.ndarray:
    q, alpha, s = split(packed, block)
    return (code_values(code)[q] * (s / alpha)[:, None]).reshape(rows, hidden)


def scale_of(u: np.ndarray, block: int, code: str) -> np.ndarray:
    """s of every block: the least 2^e, e >= -126, with max|u| <= Qmax 2^e."""
    top = np.abs(u.reshape(-1, block)).max(axis=1)
    out = np.zeros_like(top)
    for i, t in enumerate(top):
        if t > 0:
            m, e = math.frexp(t / QMAX[code])          # t / Qmax = m 2^e, m in [0.5, 1)
            e = e - 1 if math.ldexp(QMAX[code], e - 1) >= t else e
            out[i] = math.ldexp(1.0, max(e, -126))
    return out


def step_at(u: np.ndarray, s: np.ndarray, block: int, code: str) -> np.ndarray:
    """Spacing of the code grid, in units of u, around every element."""
    v = np.abs(u.reshape(-1, block)) / np.where(s == 0, 1, s)[:, None]
    if code == "int8":
        step = np.ones_like(v)
    else:
        m_bits, e_min = MANTISSA[code]
        e = np.floor(np.log2(np.maximum(v, 2.0 ** e_min)))
        step = 2.0 ** (e - m_bits)
    return (step * s[:, None]).reshape(u.shape)


def encode(u: np.ndarray, block: int, code: str):
    """Values (on the grid, nearest, ties to even) and scales of u."""
    s = scale_of(u, block, code)
    step = step_at(u, s, block, code)
    v = np.divide(u, step, out=np.zeros_like(u), where=step > 0)
    return np.rint(v) * step, s


def make_records(u: torch.Tensor, block: int, code: str) -> torch.Tensor:
    """A packed buffer of u (CPU tensor), power-of-two scales."""
    w = f64(u)
    values, s = encode(w, block, code)
    table = code_values(code)
    order = np.argsort(np.where(np.isfinite(table), table, np.inf), kind="stable")
    grid = table[order][np.isfinite(table[order])]
    v = np.divide(values.reshape(-1, block), s[:, None], out=np.zeros((s.size, block)), where=s[:, None] > 0)
    at = np.searchsorted(grid, v)
    q = order[at].astype(np.uint8)
    assert np.array_equal(table[q], v)
    tail = np.stack([np.ones_like(s), s], 1).astype("<f4").view(np.uint8)
    return torch.from_numpy(np.concatenate([q, tail], 1).reshape(-1).copy())


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

def layernorm(h: np.ndarray, weight, bias, eps: float):
    """y, mean, rstd, xhat and the bound on xhat's error."""
    mean = h.mean(1)
    centred = h - mean[:, None]
    rstd = 1 / np.sqrt((centred ** 2).mean(1) + eps)
    xhat = centred * rstd[:, None]
    y = xhat * (1 if weight is None else weight) + (0 if bias is None else bias)
    d = depth(h.shape[1])
    off_mean = d * U32 * np.abs(h).mean(1)
    # rstd: half of the variance's relative error (the sum, and the shift of the centre), plus the root and division
    off_rstd = rstd * ((d + 16) * U32 + (off_mean * rstd) ** 2 + off_mean * rstd * np.abs(xhat).mean(1) * (d * U32))
    off_xhat = (off_mean * rstd)[:, None] + np.abs(centred) * off_rstd[:, None] + 4 * U32 * (
        np.abs(xhat) + (np.abs(mean) * rstd)[:, None])
    return y, mean, rstd, xhat, off_mean, off_rstd, off_xhat


def layernorm_grads(dy, xhat, rstd, weight, off_xhat=0.0):
    """dx, dweight, dbias and the bounds on their 32-bit errors."""
    a = dy * (1 if weight is None else weight)
    c1, ax = a.mean(1, keepdims=True), (a * xhat)
    c2 = ax.mean(1, keepdims=True)
    r = rstd[:, None]
    dx = r * (a - c1 - xhat * c2)
    d = depth(dy.shape[1])
    off_c1 = d * U32 * np.abs(a).mean(1, keepdims=True)
    off_c2 = (d + 4) * U32 * np.abs(ax).mean(1, keepdims=True) + (np.abs(a) * off_xhat).mean(1, keepdims=True)
    off_dx = r * (off_c1 + np.abs(xhat) * off_c2 + np.abs(c2) * off_xhat
                  + 8 * U32 * (np.abs(a) + np.abs(c1) + np.abs(xhat * c2)))
    rows = dy.shape[0]
    off_dw = (rows + 16) * U32 * np.abs(dy * xhat).sum(0) + (np.abs(dy) * off_xhat).sum(0)
    off_db = (rows + 16) * U32 * np.abs(dy).sum(0)
    return dx, (dy * xhat).sum(0), dy.sum(0), off_dx, off_dw, off_db


# ---------------------------------------------------------------------------
# GELU
# ---------------------------------------------------------------------------

_A, _B = math.sqrt(2 / math.pi), 0.044715


def gelu(u: np.ndarray, tanh_form: bool):
    """gelu(u) and its slope."""
    if tanh_form:
        v = _A * (u + _B * u ** 3)
        t = np.tanh(v)
        return 0.5 * u * (1 + t), 0.5 * (1 + t) + 0.5 * u * (1 - t ** 2) * _A * (1 + 3 * _B * u ** 2)
    cdf = 0.5 * _erfc(-u / math.sqrt(2))
    return u * cdf, cdf + u * np.exp(-u * u / 2) / math.sqrt(2 * math.pi)


def gelu_bound(u: np.ndarray) -> np.ndarray:
    """32-bit error of gelu(u): Phi(u) in [0, 1] to eight roundings, times u."""
    return 8 * U32 * np.abs(u)


def slope_bound(u: np.ndarray) -> np.ndarray:
    """32-bit error of the slope: Phi(u), and u phi(u) whose exponent's rounding
    weighs u^2 / 2 times (u^2 |u| phi(u) <= 1, and u^4 phi-like terms of the tanh form stay below 4)."""
    return 16 * U32 * (1 + np.minimum(np.abs(u), 4))


def within(got: torch.Tensor, want: np.ndarray, off, kind=None, what=""):
    """|got - want| <= off plus one rounding to got's type, element by element."""
    kind = kind or got.dtype
    g = f64(got)
    bound = off + UNIT[kind] * (np.abs(want) + off) + TINY[kind]
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} elements off, worst "
                           f"{np.max(np.abs(g - want) / bound):.3g} times the bound")
