"""Oracle: RMS norm of query / key heads and rotation by position, float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages fix position ids (a packed token keeps the position it has in its
own sequence); the norm and the rotation are the standard ones: for a head
vector x at position t,

    n = x * w / sqrt(mean(x^2) + eps)
    pair (a, b) of n -> complex n_a + i n_b times exp(i * inv_freq * t)

over pairs (c, c + rot / 2), or (2c, 2c + 1) when interleaved; channels from
``rot`` on pass as n.
"""
from __future__ import annotations

import numpy as np


def _pairs(rot: int, interleaved: bool):
    c = np.arange(rot // 2)
    return (2 * c, 2 * c + 1) if interleaved else (c, c + rot // 2)


def _turn(n: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, rot: int, interleaved: bool, sign: float) -> np.ndarray:
    out = n.copy()
    if rot:
        a, b = _pairs(rot, interleaved)
        ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
        z = (n[..., a] + 1j * n[..., b]) * np.exp(1j * sign * ang)[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def forward(x, w, pos, inv_freq, rot, interleaved=False, eps=1e-6) -> np.ndarray:
    """x [N, H, D], w [D], pos [N], inv_freq [rot / 2] -> y [N, H, D]."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    n = x * w / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(n, pos, inv_freq, rot, interleaved, 1.0)


def backward(x, w, pos, inv_freq, rot, dy, interleaved=False, eps=1e-6):
    """Gradients (dx [N, H, D], dw [D]) of sum dy . y, written out from the
    quotient x / sqrt(mean(x^2) + eps)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    dn = _turn(np.asarray(dy, np.float64), pos, inv_freq, rot, interleaved, -1.0)
    s = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (dn * x / s).sum((0, 1))
    u = dn * w
    return u / s - x * (u * x).sum(-1, keepdims=True) / (x.shape[-1] * s ** 3), dw
