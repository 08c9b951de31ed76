"""Exact phases for the rotary tests: positions times frequencies in integers, 1 / (2 pi) to 700 bits."""
from __future__ import annotations

import math

import numpy as np

BITS = 700


def _inv_two_pi() -> int:
    """floor(2^BITS / (2 pi)) give or take a few, by Machin's formula for pi."""
    one = 1 << (BITS + 40)

    def arctan_inv(n):
        total = term = one // n
        k, sign = 1, -1
        while term:
            term //= n * n
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total
    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    return (one * one // (2 * pi)) >> 40


INV_TWO_PI = _inv_two_pi()


def turns(position: int, freq: float) -> int:
    """position * freq / (2 pi) modulo 1, in units of 2^-400 (freq is taken exactly)."""
    num, den = float(freq).as_integer_ratio()
    return ((position * num * INV_TWO_PI) // den >> (BITS - 400)) % (1 << 400)


def angle(position: int, freq: float) -> float:
    t = turns(position, freq)
    return 2 * math.pi * ((t >> 300) / 2.0 ** 100)


def rope(x: np.ndarray, positions, inv_freq) -> np.ndarray:
    """x [T, H, 256] with adjacent pairs, one axis, every angle reduced exactly; float64."""
    y = np.array(x, dtype=np.float64)
    for i, f in enumerate(inv_freq):
        a = np.array([angle(int(p), float(f)) for p in positions])
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        u, w = x[..., 2 * i].astype(np.float64), x[..., 2 * i + 1].astype(np.float64)
        y[..., 2 * i], y[..., 2 * i + 1] = u * c - w * s, w * c + u * s
    return y
