"""4-bit attention at scores of 2^10 to 2^30, where a float32 score holds few or no bits below one."""
import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from oracle import fp4
from tests import fp4_util as fu

pytestmark = pytest.mark.gpu

# name, [(q_len, L)], q heads, the path, the bits of the kernel that serves it
KERNELS = [
    ("verify", [(4, 500), (2, 77), (4, 5000)], 16, 0, 2),
    ("verify, planned before", [(4, 500), (2, 77), (4, 5000)], 16, 3, 2),
    ("prefill", [(150, 400), (40, 3000)], 8, 0, 4),
    ("single tokens", [(1, 300), (1, 17), (1, 4000)], 8, 0, 128),
    ("warp level", [(4, 500), (40, 300)], 8, 1, 8),
]


def _run(c, path, bit):
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    prev = pg.paged_gqa_set_path(path)
    try:
        pg.paged_gqa_attn_fp4(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out)
    finally:
        pg.paged_gqa_set_path(prev)
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()
    assert pg.paged_gqa_last_plan()["path_bits"] & bit
    return out


def _alone(c):
    """Per row (token, head): is its best key's weight all there is? float32 sums of 256 products are off by at
    most 2^-16 of the sum of their sizes, here below 2^4 times the row's largest score, so a key that
    trails by 13 + 2^-11 of that score (log2 units) weighs less than 2^-13 whatever the rounding."""
    k = fp4.values(*fp4.unpack(c.k.cpu().numpy(), False))[:, :, 0]
    q, table, qsl = c.q.double().cpu().numpy(), c.table.cpu().numpy(), c.qsl.cpu().numpy()
    alone = []
    for s, (qn, L) in enumerate(c.seqs):
        keys = k[table[s, :-(-L // c.page)]].reshape(-1, 256)[:L] * (c.kd * c.scale / np.log(2))
        for t in range(qn):
            x = q[qsl[s] + t] @ keys[:L - qn + t + 1].T
            size = np.abs(q[qsl[s] + t]) @ np.abs(keys[:L - qn + t + 1]).T
            best = np.sort(x, -1)
            gap = best[:, -1] - best[:, -2] if x.shape[-1] > 1 else np.full(len(x), np.inf)
            assert (size.max(-1) < 16 * np.abs(x).max(-1)).all()
            alone.append(gap > 13 + 2.0 ** -11 * np.abs(x).max(-1))
    return np.concatenate(alone)


@pytest.mark.parametrize("sign,bits", [(0, 30), (1, 30), (-1, 30), (0, 10), (0, 14), (1, 14), (-1, 18), (0, 24)])
@pytest.mark.parametrize("i", range(len(KERNELS)), ids=[k[0] for k in KERNELS])
def test_large_scores_pick_the_best_key(i, sign, bits):
    """Scores of either sign, all positive, all negative; every fourth head's are of ordinary size.

    The rows compared: the ordinary ones and those whose best key has all the weight."""
    name, seqs, hq, path, bit = KERNELS[i]
    c = fu.make(seqs, hq, 1, 16, seed=300 + i)
    if sign:
        held = c.k[..., :128]
        c.k[..., :128] = held & 0x77  # every code positive
        c.q = c.q.abs() * sign
    size = torch.full((1, hq, 1), 2.0 ** bits)
    size[:, 1::4] = 1.0
    c.q = (c.q.float().cpu() * size).bfloat16().cuda()
    out = _run(c, path, bit)
    assert bool(out.isfinite().all())
    ordinary = np.tile(np.arange(hq) % 4 == 1, c.T)
    rows = np.flatnonzero(ordinary | _alone(c))
    assert len(rows) > 0.8 * c.T * hq
    fu.check(c, out, name, rows=rows)


@pytest.mark.parametrize("bits", [13, 30])
@pytest.mark.parametrize("name,seqs,hq,path,bit", [
    ("verify", [(4, 500)], 16, 0, 2),
    ("prefill", [(16, 500)], 8, 0, 4),
    ("single token", [(1, 250)], 8, 0, 128),
    ("warp level", [(4, 500)], 16, 1, 8),
])
def test_equal_keys_share_a_row_evenly_however_large_their_score(name, seqs, hq, path, bit, bits):
    """One key in every slot: the output is the mean of the V that a token sees (in one piece: the sums of
    pieces meet through their logarithms, which a float32 next to 2^30 does not hold)."""
    c = fu.make(seqs, hq, 1, 16, seed=320)
    c.k[:] = c.k[int(c.table[0, 0]), 0, 3].clone()
    c.q = (c.q.float() * 2.0 ** bits).bfloat16()
    fu.check(c, _run(c, path, bit), name)


@pytest.mark.parametrize("scale,kd", [(0.0, 0.01), (-1.0 / 16, 0.01), (0.4, 0.01), (1.0 / 16, -0.02), (2.0 ** -40, 2.0 ** 30), (1e-30, 0.01)])
@pytest.mark.parametrize("i", range(len(KERNELS)), ids=[k[0] for k in KERNELS])
def test_other_scales(i, scale, kd):
    """A scale of zero (the mean of the V seen), negative ones, scales far from one."""
    name, seqs, hq, path, bit = KERNELS[i]
    c = fu.make(seqs, hq, 1, 16, seed=350 + i)
    c.scale, c.kd = scale, kd
    fu.check(c, _run(c, path, bit), name)
