"""Oracle: rotary positions in fp64 (test infrastructure only; see the package
docstring)."""
from __future__ import annotations

import numpy as np


def rotate(x, positions, frequencies, factor=1.0, interleaved=False):
    """x [tokens, heads, d]; the first 2 len(frequencies) elements of each head
    are turned by positions * frequencies, the others passed on."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    rot = 2 * len(frequencies)
    a = np.asarray(positions, np.float64)[:, None, None] * np.asarray(frequencies, np.float64)
    i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., i] = factor * (x[..., i] * np.cos(a) - x[..., j] * np.sin(a))
    y[..., j] = factor * (x[..., j] * np.cos(a) + x[..., i] * np.sin(a))
    return y
