"""Rotary positions at frequencies of every size, against exactly reduced angles."""
import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import rope_util as ru

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("freqs", [
    [1e-40, 1e-30, 3e-9, 1e-3, 0.5, 1.0, 6.2831855, 1234.567, 3e7, 2e-45, 0.0, 1e10, 1e-7, 0.1, 2.0, 31.4],
    [1e5, 1e6, 1e8, 1e9, 1e12, 1e15, 1e18, 1e21, 1e25, 1e30, 1e34, 3.4028235e38, -1e5, -1e10, -3e30, 16777216.0],
])
def test_frequencies_of_every_size_keep_their_phase(freqs):
    inv = torch.tensor(freqs, dtype=torch.float32).cuda()
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 2 ** 20, 7]], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 2, 256, generator=g).bfloat16().cuda()
    out, kout = torch.empty_like(x), torch.empty_like(x)
    pg.paged_gqa_rope(x, x, pos, inv, [16], out, kout, adjacent=True)
    assert bool((out == kout).all())
    xs = x.double().cpu().numpy()
    ref = ru.rope(xs, pos[0].tolist(), inv.tolist())
    # bf16 once: 2^-8 of the value; the fp32 phase (2^-25 turns, 2 pi of it), cosine, sine, products and their
    # sum: below 2^-20 of the pair's size, which is below 8
    off = np.abs(out.double().cpu().numpy() - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * 8)
    for i, f in enumerate(freqs):
        assert (off[..., 2 * i:2 * i + 2] <= 0).all(), f"frequency {f}"
