"""Token counts that do not fit the tensors: the 4-bit cache's write and read stay inside them, flag the call
and leave everything else as it was. (The tensors here are the first rows of larger ones.)"""
import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from oracle import fp4
from tests import fp4_util as fu

pytestmark = pytest.mark.gpu

BOUNDS = -5

# query_start_loc against T = 8, and which sequences keep their tokens
STARTS = [
    ("ends beyond T", [0, 3, 17], [True, False]),
    ("one token too many", [0, 3, 9], [True, False]),
    ("far beyond T", [0, 3, 2 ** 31 - 1], [True, False]),
    ("begins before 0", [-2, 3, 8], [False, True]),
    ("ends before T", [0, 3, 6], [True, True]),
    ("begins after 0", [2, 3, 8], [True, True]),
]


def _case(hkv=2):
    c = fu.make([(3, 30), (20, 116)], hkv, hkv, 16, seed=330)
    return c, 8


@pytest.mark.parametrize("name,starts,valid", STARTS, ids=[s[0] for s in STARTS])
def test_write(name, starts, valid):
    c, T = _case()
    g = torch.Generator().manual_seed(1)
    kn, vn = [torch.randn(T + 40, 2, 256, generator=g).bfloat16().cuda() for _ in range(2)]
    want = [c.k.cpu().numpy(), c.v.cpu().numpy()]
    for s in range(2):
        a, b = starts[s], min(starts[s + 1], T)
        if valid[s]:
            new = [x[a:b].float().cpu().numpy() for x in (kn, vn)]
            want = fp4.write(*new, *want, c.table[s:s + 1].cpu().numpy(), c.lens[s:s + 1].cpu().numpy(),
                             np.array([0, b - a]), c.kd, c.vd)
    qsl = torch.tensor(starts, dtype=torch.int32, device="cuda")
    pg.paged_gqa_cache_write_fp4(kn[:T], vn[:T], c.k, c.v, c.table, c.lens, qsl, c.kd, c.vd)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    assert (c.k.cpu().numpy() == want[0]).all() and (c.v.cpu().numpy() == want[1]).all()


@pytest.mark.parametrize("name,starts,valid", STARTS, ids=[s[0] for s in STARTS])
def test_read(name, starts, valid):
    c, T = _case()
    out = torch.full((2, T + 40, 2, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    qsl = torch.tensor(starts, dtype=torch.int32, device="cuda")
    pg.paged_gqa_cache_read_fp4(c.k, c.v, c.table, c.lens, qsl, c.kd, c.vd, out[0, :T], out[1, :T])
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    assert bool((out[:, T:] == 3.0).all())
    want = np.zeros((2, T, 2, 256))
    for s in range(2):
        a, b = starts[s], min(starts[s + 1], T)
        if valid[s]:
            want[:, a:b] = fp4.read(c.k.cpu().numpy(), c.v.cpu().numpy(), c.table[s:s + 1].cpu().numpy(),
                                    c.lens[s:s + 1].cpu().numpy(), np.array([0, b - a]), c.kd, c.vd)
    got = out[:, :T].double().cpu().numpy()
    # one rounding to fp32 (2^-24) and one to bf16 (2^-8, which is half a step)
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()
