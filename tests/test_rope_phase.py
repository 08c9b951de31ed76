"""The rotary kernel's fixed-point phase in Python integers: off by less than 2^-31 turns for every finite
frequency and every 32-bit position."""
import os
import random
import re
import struct

import numpy as np

import paged_gqa_gb300
from tests import rope_util as ru


def _words():
    src = open(os.path.join(os.path.dirname(paged_gqa_gb300.__file__), "csrc", "rope.cu")).read()
    return [int(w, 16) for w in re.findall(r"0x([0-9a-f]{8})u", re.search(r"kInv2Pi\[7\] = \{([^}]*)\}", src).group(1))]


def _turns_of(x, words):
    """rope.cu's turns_of: |x| = m 2^e, 96 bits of 1 / (2 pi) from bit max(e, 0) on."""
    b = struct.unpack("<I", struct.pack("<f", x))[0]
    be = b >> 23 & 0xFF
    m, e = (b & 0x7FFFFF) | (0x800000 if be else 0), (be or 1) - 150
    c = sum(w << 32 * (6 - i) for i, w in enumerate(words))
    window = c >> (224 - max(e, 0) - 96) & (1 << 96) - 1
    f = m * window >> 32 + max(-e, 0) & (1 << 64) - 1
    return -f % (1 << 64) if b >> 31 else f


def test_the_constant():
    assert sum(w << 32 * (6 - i) for i, w in enumerate(_words())) == ru.INV_TWO_PI >> (ru.BITS - 224)


def test_phases_of_all_sizes_of_frequencies():
    words, rng = _words(), random.Random(1)
    freqs = [1.0, 1e5, 3e7, 1e10, 1e20, 3.4028235e38, 2.0 ** -149, 2.0 ** -126, 6.2831855, 10000.0 ** -0.75]
    freqs += [rng.uniform(1, 2) * 2.0 ** rng.randint(-149, 126) for _ in range(3000)]
    for f in freqs:
        f = float(np.float32(f)) * rng.choice([1, -1])
        for p in (1, -1, 2 ** 31 - 1, -2 ** 31, rng.randint(-2 ** 31, 2 ** 31 - 1)):
            phase = p * _turns_of(f, words) >> 32 & 0xFFFFFFFF
            off = ((phase << 368) - ru.turns(p, f) + (1 << 399)) % (1 << 400) - (1 << 399)
            assert abs(off) < 1 << 369, (f, p, off / 2.0 ** 369)
