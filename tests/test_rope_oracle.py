"""The rotary oracle against complex rotations and closed forms."""
import numpy as np
import pytest

from oracle import rope as ro


def test_axis_maps():
    assert ro.axes_of([2, 1, 1], False) == [0, 0, 1, 2]
    assert ro.axes_of([4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert ro.axes_of([3, 3, 2], True) == [0, 1, 2, 0, 1, 2, 0, 1]
    for sections in ([24, 20, 20], [11, 11, 10], [8], [4, 4]):
        for il in (False, True):
            a = ro.axes_of(sections, il)
            assert [a.count(i) for i in range(len(sections))] == sections


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_is_complex_multiplication_and_keeps_norms(adjacent):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 256))
    pos = rng.integers(-1000, 1000, (2, 5))
    inv = (10000.0 ** -(np.arange(0, 64, 2) / 64)).astype(np.float32)
    y = ro.rope(x, pos, inv, [16, 16], False, adjacent)
    assert (y[..., 64:] == x[..., 64:]).all()
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if adjacent else (slice(0, 32), slice(32, 64))
    ang = np.concatenate([pos[0][:, None] * inv[:16].astype(np.float64), pos[1][:, None] * inv[16:].astype(np.float64)], 1)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang)[:, None]
    assert np.allclose(y[..., a], z.real, atol=1e-11) and np.allclose(y[..., b], z.imag, atol=1e-11)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    back = ro.rope(y, -pos, inv, [16, 16], False, adjacent)
    assert np.allclose(back, x, atol=1e-11)
