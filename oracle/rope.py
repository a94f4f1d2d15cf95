"""Norms and rotation of query and key rows, and the keys' move to new positions (fp64).

A pair (a, b) is the complex number a + i b; it is multiplied by exp(i t), t = position * inverse frequency."""
from __future__ import annotations

import numpy as np

__all__ = ["rope_freqs", "rope_rows"]


def rope_freqs(rot, theta):
    return np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])


def rope_rows(x, pos, freqs, axes=None, adjacent=False, weight=None, eps=0.0, scale=1.0):
    """x [n][H][d], pos [n_axis][n] (or [n][H] positions of single rows), freqs [pairs], axes [pairs].

    Returns (y, mag): mag is the length |a| + |b| that an error of the angle or of the norm moves y by (|y| where
    nothing turns)."""
    x = np.array(x, np.float64)
    n, h, d = x.shape
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    m = len(freqs)
    pos = np.asarray(pos)
    y, mag = x.copy(), np.abs(x)
    for i in range(m):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + m)
        p = pos if pos.shape == (n, h) and axes is None else pos[0 if axes is None else axes[i]][:, None]
        z = (x[:, :, a] + 1j * x[:, :, b]) * np.exp(1j * (p.astype(np.float64) * freqs[i])) * scale
        y[:, :, a], y[:, :, b] = z.real, z.imag
        mag[:, :, a] = mag[:, :, b] = (np.abs(x[:, :, a]) + np.abs(x[:, :, b])) * scale
    return y, mag
