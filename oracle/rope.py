"""Oracle: rotary positions in all the forms that can be served.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Readings (the pages do not print the rotation): pair i of a head's first `dim` elements turns by
t * f_i, f_i = base^(-2i/dim); the pair is (x_i, x_{i + dim/2}), or (x_2i, x_{2i+1}) where
interleaved.  For long contexts: "linear" divides every f_i; "ntk" changes the base so that the
slowest pair is divided by factor and the fastest stays; "parts" divides only what turns less
than `low` times within the original context, keeps what turns more than `high` times, with a
ramp between.
"""
import math

import numpy as np


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0,
                high=4.0):
    """Radians per position of the dim/2 pairs."""
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    out = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "parts":
            turns = original_len * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out)


def turn(x, pos, freqs, interleaved=False, magnitude=1.0):
    """x [T, H, D], positions pos [T] -> the turned rows."""
    y = np.array(x, dtype=np.float64, copy=True)
    n = len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        u = np.asarray(pos, dtype=np.float64) * f
        c, s = magnitude * np.cos(u)[:, None], magnitude * np.sin(u)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y
