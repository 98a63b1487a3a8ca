"""Plain 64-bit implementations of the 8-bit projections, the quantisation of their operands
and the rotary positions, for their tests.  Written from the formulas in include/hyena.h
with numpy; they share no code with the kernels."""
from __future__ import annotations

import math

import numpy as np

from tests.serving_ref import decode

RUN = 128


def widen(codes, scale, rows=1):
    """Codes (n, k) times the scales (n), (n, runs), or (row blocks, runs) with rows = 128."""
    v = decode(codes)
    s = np.asarray(scale, dtype=np.float64)
    if s.ndim == 1:
        return v * s[:, None]
    n, k = v.shape
    r, c = np.arange(n) // rows, np.arange(k) // RUN
    return v * s[r[:, None], c[None, :]] if k else v


def product(x, xs, w, ws):
    """(y, size): y = x w^T and the sums of the magnitudes behind each element."""
    a, b = widen(x, xs), widen(w, ws, RUN)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def act(g, kind):
    if kind == "gelu":
        return g * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-g / math.sqrt(2.0))
    with np.errstate(over="ignore"):
        if kind == "gelu_tanh":
            return g / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        if kind == "silu":
            return g / (1 + np.exp(-g))
    return g


def block_scales(x, rows, cols):
    """max|x| / 448 of each block (1 where it is 0), and the scale of each element."""
    n, k = x.shape
    rows, cols = rows or n, cols or k
    out = np.ones((-(-n // rows), -(-k // cols)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            m = np.abs(x[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols]).max()
            if m > 0:
                out[i, j] = max(m / 448, 2.0 ** -140)
    return out, np.repeat(np.repeat(out, rows, 0)[:n], cols, 1)[:, :k]


def rope(x, positions, inv_freq, interleaved, eps=None, weight=None):
    """(y, size): the turned heads, and |a| + |b| (or |x|) of the values that each came from."""
    T, H, DH = x.shape
    x = x.astype(np.float64).copy()
    if eps is not None:
        top = np.maximum(np.abs(x).max(-1, keepdims=True), 1e-300)
        z = x / top
        x = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps / top / top)
        if weight is not None:
            x = x * weight
    y, size = x.copy(), np.abs(x)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        f = positions.astype(np.float64) * float(inv_freq[i])
        c, s = np.cos(f)[:, None], np.sin(f)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    return y, size
