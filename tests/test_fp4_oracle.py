"""The 4-bit cache's oracle against its definition."""
import numpy as np
import torch

from oracle import fp4


def test_every_code_and_scale_decodes():
    want = [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert fp4.code_value(np.arange(16)).tolist() == want + [-x for x in want]
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = fp4.scale_value(np.arange(256))
    assert ((got == ref) | (np.isnan(got) & np.isnan(ref))).all()


def test_encoding_rounds_to_the_nearest_level_and_ties_to_even_codes():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 6.0: 7, 100.0: 7, np.inf: 7}
    for x, c in ties.items():
        assert fp4.encode(np.float32(x)) == c and fp4.encode(np.float32(-x)) == c + 8, x
    assert fp4.encode(np.float32("nan")) == 7
    x = np.random.default_rng(0).uniform(-8, 8, 20000).astype(np.float32)
    got = fp4.code_value(fp4.encode(x))
    near = np.abs(x[:, None].astype(np.float64) - np.concatenate([-fp4.LEVELS, fp4.LEVELS])).min(1)
    assert (np.abs(got - x) == near).all()


def test_quantise_keeps_levels_and_marks_nans():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (50, 256)).astype(np.uint8)
    codes[:, ::16] = 7  # each group reaches 6, so its scale is found again
    s8 = rng.integers(0x10, 0x70, (50, 16)).astype(np.uint8)
    x = fp4.values(codes, s8).astype(np.float32)
    c2, s2 = fp4.quantise(x, 1.0)
    assert (s2 == s8).all() and (fp4.code_value(c2) == fp4.code_value(codes)).all()
    x[3, 20] = np.nan
    x[4, 40] = np.inf
    x[5, :16] = 0
    c2, s2 = fp4.quantise(x, 1.0)
    assert s2[3, 1] == 0x7F and s2[4, 2] == 0x7E and s2[5, 0] == 0
    assert np.isnan(fp4.values(c2, s2)[3, 16:32]).all()
    assert (fp4.values(c2, s2)[5, :16] == 0).all() and fp4.values(c2, s2)[4, 40] == 448 * 6


def test_packing_against_single_values():
    rng = np.random.default_rng(2)
    NB, P, H = 3, 32, 2
    codes = rng.integers(0, 16, (NB, P, H, 256)).astype(np.uint8)
    s8 = rng.integers(0, 127, (NB, P, H, 16)).astype(np.uint8)
    for is_v in (False, True):
        c = fp4.pack(codes, s8, is_v)
        assert c.shape == (NB, H, P, 144)
        u = fp4.unpack(c, is_v)
        assert (u[0] == codes).all() and (u[1] == s8).all()
        one = np.zeros_like(c)
        for n in range(NB):
            for t in range(P):
                for h in range(H):
                    fp4.put(one, n, h, t, is_v, codes[n, t, h], s8[n, t, h])
        assert (one == c).all()
        # single bytes, by the definition
        flat = c[1, 1].reshape(-1)
        t, i, g = 21, 77, 9
        at = t * 144 + i if not is_v else 16 * 144 + i * 16 + 5
        assert flat[at] == codes[1, t, 1, 2 * i] | codes[1, t, 1, 2 * i + 1] << 4
        at = t * 144 + 128 + g if not is_v else 16 * 144 + 2048 + g * 16 + 5
        assert flat[at] == s8[1, t, 1, g]
