"""Oracle: what an activation checkpoint in 8 bits keeps, float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

For 32 successive channels of a token with largest magnitude a, s is the
smallest power of two from 2^-117 on with a <= 448 s, and a value keeps
x / s to the nearest e4m3 number (ties to even): four significant bits from
2^-6 on, steps of 2^-9 below.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 number of |v| <= 448, ties to even."""
    _, e = np.frexp(v)                       # v = f 2^e, 1/2 <= |f| < 1
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(v / step) * step          # rint: ties to even


def scales(x: np.ndarray) -> np.ndarray:
    """Scale of every block of channels, [N, blocks]; NaN where it holds an infinity or a NaN."""
    n, c = x.shape
    x = np.pad(np.abs(np.asarray(x, np.float64)), ((0, 0), (0, -c % BLOCK))).reshape(n, -1, BLOCK)
    top = x.max(-1) if x.size else np.zeros(x.shape[:2])
    bad = ~np.isfinite(top)
    f, e = np.frexp(np.where(bad, 1.0, top) / 448)
    s = np.ldexp(1.0, np.maximum(np.where(f == 0.5, e - 1, e), -117))
    s[np.where(bad, 1.0, top) == 0] = 2.0 ** -117
    return np.where(bad, np.nan, s)


def keep(x: np.ndarray) -> np.ndarray:
    """What is restored of x [N, C], as a float32 holds it: a magnitude that rounds to 2^128 is an infinity."""
    s = np.repeat(scales(x), BLOCK, axis=1)[:, :x.shape[1]]
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(np.isnan(s), np.nan, e4m3(np.where(np.isnan(s), 0.0, np.asarray(x, np.float64) / s)) * s)
        return y.astype(np.float32).astype(np.float64)
