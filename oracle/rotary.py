"""Rotary positions in float64, pair by pair (NumPy).  Test infrastructure only (see the package docstring)."""

import numpy as np


def rotary(x, positions, inv_freq, layout, start=0, scale=1.0, inverse=False):
    """x float64 [N0, N1, H, D]; positions int [N0, N1]; inv_freq float64 [rot/2]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for p, f in enumerate(np.asarray(inv_freq, dtype=np.float64)):
        a, b = (p, p + half) if layout == "half" else (2 * p, 2 * p + 1)
        a, b = start + a, start + b
        angle = np.asarray(positions, dtype=np.float64) * f
        c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
        if inverse:
            s = -s
        y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
        y[..., b] = scale * (x[..., b] * c + x[..., a] * s)
    return y
