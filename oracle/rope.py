"""CPU oracle for the rotary positions: fp64 from the definition.  TEST INFRASTRUCTURE ONLY;
imports nothing from the product path.

A pair (a, b) at position p becomes mscale (a cos t - b sin t, b cos t + a sin t) with
t = p * inv_freq[j]; written here as the product of a + ib with mscale e^{it}.  The gradient
multiplies with the conjugate.  Pairs: columns (j, j + rot/2), or (2j, 2j + 1) interleaved;
columns from rot on are unchanged.
"""
from __future__ import annotations

import numpy as np


def rotate(x, inv_freq, positions, interleaved: bool, mscale: float, backward: bool = False) -> np.ndarray:
    """x [B, H, N, d] values, inv_freq [rot/2], positions [B, N] -> fp64 [B, H, N, d]."""
    x = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    half = f.size
    t = np.asarray(positions, dtype=np.float64)[:, None, :, None] * f
    w = mscale * np.exp((-1j if backward else 1j) * t)
    a, b = (np.s_[..., 0:2 * half:2], np.s_[..., 1:2 * half:2]) if interleaved else (np.s_[..., :half], np.s_[..., half:2 * half])
    z = (x[a] + 1j * x[b]) * w
    x[a], x[b] = z.real, z.imag
    return x
