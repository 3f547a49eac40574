"""fp64 oracle of the rotary positions, written from the definition in
``include/nvfp4.h`` alone."""
from __future__ import annotations

import numpy as np


def rope(x, positions, freqs, axis=None, adjacent=False, factor=1.0):
    """x [tokens, heads, dim], positions [axes, tokens], freqs [pairs] -> (the rotated
    rows, and for error bounds factor * (|a| + |b|) of each element's pair, and the
    largest |angle| of the call), float64."""
    x = np.asarray(x, np.float64)
    pairs = len(freqs)
    out, size, far = x.copy(), np.abs(x), 0.0
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + pairs)
        k = 0 if axis is None else int(axis[i])
        pos = positions[k] if k < len(positions) else np.zeros(x.shape[0])
        t = np.asarray(pos, np.float64) * freqs[i]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        with np.errstate(invalid="ignore"):
            out[:, :, a] = factor * (x[:, :, a] * c - x[:, :, b] * s)
            out[:, :, b] = factor * (x[:, :, b] * c + x[:, :, a] * s)
            size[:, :, a] = size[:, :, b] = factor * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
        far = max(far, float(np.abs(t).max(initial=0)))
    return out, size, far
