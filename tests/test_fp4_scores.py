"""The arithmetic of the 4-bit attention's exponents at scores of any size, in float32 steps on the CPU.

x = rn(rn(s c) + rn(sigma - m)), m the largest rn(s c): what the softmax of the tcgen05 kernel takes 2^x of
after it has moved a row's reference. It has to be at most tau + sigma, the limit of its vote, or the row
would ask for a new reference again, and 2^x has to fit f16.
"""
import os
import re

import numpy as np
import pytest

import paged_gqa_gb300

F = np.float32


def _constants():
    src = open(os.path.join(os.path.dirname(paged_gqa_gb300.__file__), "csrc", "fp4_tc.cu")).read()
    return [F(re.search(rf"constexpr float {n} = ([0-9.]+)f;", src).group(1)) for n in ("kTau", "kSigma")]


def _exponents(s, c, sigma):
    """Rows of scores s and their scales c (float32) -> x by rounded products, and by fused ones."""
    p = s * c                                  # float32: rounded
    m = p.max(-1, keepdims=True)
    mo = sigma - m
    exact = s.astype(np.float64) * c.astype(np.float64)   # 48 bits: exact
    return p + mo, (exact + mo.astype(np.float64)).astype(F)


@pytest.mark.parametrize("sign", [0, 1, -1])
def test_one_new_reference_is_enough_for_scores_of_any_size(sign):
    tau, sigma = _constants()
    rng = np.random.default_rng(3)
    for e in range(-20, 121):
        s = rng.standard_normal((64, 128)).astype(F)
        s = sign * np.abs(s) if sign else s
        c = (rng.uniform(0.5, 1, (64, 1)) * 2.0 ** e).astype(F)
        x, _ = _exponents(s.astype(F), c, sigma)
        assert (x <= tau + sigma).all() and (x.max(-1) >= 0).all(), e


def test_the_bound_at_every_step_around_its_worst_sizes():
    """Between 2^20 and 2^30 the rounding of sigma - m grows from nothing to all of sigma."""
    tau, sigma = _constants()
    for e in range(20, 31):
        m = (F(2.0 ** e).view(np.uint32) + np.arange(-4096, 4096)).astype(np.uint32).view(F)
        for v in (m, -m):
            x = v + (sigma - v)
            assert (x <= tau + sigma).all() and (x >= 0).all(), e


def test_equal_scores_get_equal_exponents_and_fused_products_would_not_end():
    tau, sigma = _constants()
    rng = np.random.default_rng(4)
    s, c = rng.standard_normal((500, 128)).astype(F), rng.uniform(2.0 ** 29, 2.0 ** 30, (500, 1)).astype(F)
    s[:, 64:] = s[:, :64]
    x, fused = _exponents(s, c, sigma)
    assert (x[:, 64:] == x[:, :64]).all()
    assert (fused > tau + sigma).any(-1).mean() > 0.2  # such a row would vote for a new reference for ever

