"""Plain 64-bit definitions of the 8-bit operators, for the tests (numpy)."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP e4m3 by its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits, no
    infinity, NaN at 0x7f and 0xff."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -a if c & 128 else a
    return v


VALUES = e4m3_values()


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code (ties to the even mantissa) of |v| <= 448; NaN and infinities to NaN."""
    pos = VALUES[:127]
    a = np.abs(v)
    bad = ~np.isfinite(a)
    a = np.where(bad, 0.0, a)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    c = np.where(bad, 127, c).astype(np.uint8)
    return c | np.where(np.signbit(v) & ~bad, 128, 0).astype(np.uint8)


def group_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-126 with amax / s <= 448; 1 for a group of zeros."""
    if amax == 0:
        return 1.0
    s = 2.0 ** -126
    if amax / s > 448:
        m, e = np.frexp(amax / 448)
        s = 2.0 ** (e - 1 if m == 0.5 else e)
    return s


def quantize(x: np.ndarray, layout: str):
    """x [n][rows][cols] float64 -> (codes uint8, scales float64)."""
    n, rows, cols = x.shape
    tall = 1 if layout == "rows" else BLOCK
    q = np.empty(x.shape, np.uint8)
    s = np.empty((n, -(-rows // tall), blocks(cols)))
    for i in range(n):
        for r in range(s.shape[1]):
            for c in range(s.shape[2]):
                at = (i, slice(r * tall, (r + 1) * tall), slice(c * BLOCK, (c + 1) * BLOCK))
                g = x[at]
                f = np.abs(g[np.isfinite(g)])
                s[i, r, c] = group_scale(float(f.max()) if f.size else 0.0)
                q[at] = encode(g / s[i, r, c])
    return q, s


def spread(scale: np.ndarray, rows: int, cols: int) -> np.ndarray:
    return np.repeat(np.repeat(scale, BLOCK, axis=-2), BLOCK, axis=-1)[..., :rows, :cols]


def dequantize(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """[N][K] codes and block scales -> float64."""
    return VALUES[codes] * spread(scale.astype(np.float64), *codes.shape)


def dequantize13(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """[2I][d] gate and up rows, each half with block rows of its own."""
    I, h = codes.shape[0] // 2, scale.shape[0] // 2
    return np.concatenate([dequantize(codes[:I], scale[:h]), dequantize(codes[I:], scale[h:])])


def expert(x, W13, W2):
    I = W2.shape[1]
    g, u = x @ W13[:I].T, x @ W13[I:].T
    return (g / (1.0 + np.exp(-g)) * u) @ W2.T


def moe(X, Wr, k, W13, W2, bias=None, shared=None):
    """X, Wr float64; W13, W2: expert id -> float64 matrices; shared: (Ws13, Ws2) or None; bias [B][E] or None.
    Returns out, ids (ascending), weights."""
    L = X @ Wr.T + (0.0 if bias is None else bias)
    ids = np.sort(np.argsort(-L, axis=1, kind="stable")[:, :k], axis=1)
    l = np.take_along_axis(L, ids, axis=1)
    w = np.exp(l - l.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    out = np.zeros_like(X)
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        out[t] += w[t, j][:, None] * expert(X[t], W13(e), W2(e))
    if shared is not None:
        out += expert(X, *shared)
    return out, ids, w
