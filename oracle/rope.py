"""Oracle of the rotary positions (TEST INFRASTRUCTURE ONLY): the rotation in float64, pair by pair.

Only ``tests/`` and ``__graft_entry__.smoke()`` may import this module; the CUDA library never
does, and this module never imports it.

Pair i of the first R values of a head turns by positions[axis(i), t] * inv_freq[i]. With
``interleaved`` entry i goes with axis i mod A until that axis has its number of entries, and
with axis 0 otherwise; without it the axes take consecutive runs of entries.

Parity status: pinned (tests/test_rope_oracle.py: complex rotations, inverse, norms, axis maps
written out by hand, shifts of all positions).
"""
from __future__ import annotations

import numpy as np


def axes_of(sections, interleaved: bool):
    n, A = sum(sections), len(sections)
    if not interleaved:
        return [a for a, count in enumerate(sections) for _ in range(count)]
    out, left = [], list(sections)
    for i in range(n):
        a = i % A
        if a and left[a]:
            left[a] -= 1
        else:
            a = 0
        out.append(a)
    return out


def rope(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, sections, interleaved: bool, adjacent: bool):
    """x [T, H, 256] -> float64 [T, H, 256]; inv_freq float32 (taken exactly), positions [A, T] int."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    for i, a in enumerate(axes_of(sections, interleaved)):
        # position * frequency is exact in extended precision up to 64 bits; the reduction to one
        # turn happens there, before float64 takes over
        ang = positions[a].astype(np.longdouble) * np.longdouble(inv_freq[i])
        ang = np.remainder(ang, 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))).astype(np.float64)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
        u, w = np.array(x[..., p], dtype=np.float64), np.array(x[..., q], dtype=np.float64)
        y[..., p], y[..., q] = u * c - w * s, w * c + u * s
    return y
