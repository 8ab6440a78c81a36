"""8-bit activation checkpoints by enumeration of the 8-bit values.

TEST INFRASTRUCTURE ONLY (see ``oracle/seq.py``).

A group of 128 values shares the scale 2^(E-127), E the least exponent in
[1, 254] with max <= 448 scale; a code is the nearest of the 127 magnitudes of
e4m3, the even code on a tie.  NaN and Inf have the NaN code.
"""
from __future__ import annotations

import numpy as np

GROUP = 128
# the magnitudes of codes 0 .. 126 (127 is NaN)
MAGNITUDE = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                      for c in range(127)])


def pack(x):
    """codes uint8 [R,D] and exponents uint8 [R,ceil(D/128)] of fp32-valued x [R,D]."""
    x = np.asarray(x, np.float64)
    R, D = x.shape
    code, exp = np.empty((R, D), np.uint8), np.empty((R, -(-D // GROUP)), np.uint8)
    for r in range(R):
        for j in range(exp.shape[1]):
            g = x[r, j * GROUP:(j + 1) * GROUP]
            fin = np.abs(g[np.isfinite(g)])
            top = fin.max() if fin.size else 0.0
            E = 1
            while top > 448.0 * 2.0 ** (E - 127):
                E += 1
            exp[r, j] = E
            with np.errstate(invalid="ignore"):
                v = np.abs(g) * 2.0 ** (127 - E)
            hi = np.clip(np.searchsorted(MAGNITUDE, np.where(np.isfinite(v), v, 0.0)), 1, 126)
            lo = hi - 1
            vf = np.where(np.isfinite(v), v, 0.0)
            down, up = vf - MAGNITUDE[lo], MAGNITUDE[hi] - vf
            c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
            c = np.where(np.isfinite(g), c, 127)
            code[r, j * GROUP:(j + 1) * GROUP] = c + np.where(np.signbit(g), 128, 0)
    return code, exp


def value(code, exp):
    """The numbers that codes and exponents stand for (fp64)."""
    code = np.asarray(code)
    mag = np.append(MAGNITUDE, np.nan)[code & 127]
    E = np.repeat(np.asarray(exp, np.float64), GROUP, -1)[..., :code.shape[-1]]
    return np.where(code >= 128, -mag, mag) * 2.0 ** (E - 127)
