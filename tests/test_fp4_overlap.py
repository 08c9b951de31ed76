"""Overlapping tensors that the rotary and the 4-bit cache calls refuse: host side, no GPU needed.
(Their neighbours, which they take, are tested on the GPU: such calls launch.)"""
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import test_fp4_abi as ab
from tests.test_abi import FakeTensor


def _rope(**over):
    a = dict(q=ab._at((8, 16, 256), 0), k=ab._at((8, 2, 256), 1 << 18), qo=ab._at((8, 16, 256), 1 << 19),
             ko=ab._at((8, 2, 256), 3 << 18))
    a.update(over)
    return ab._rope(**a)


def _words(shape, offset, dtype, stride=None):
    return FakeTensor(shape, dtype, ptr=(1 << 24) + offset, stride=stride)


END = 2 * 8 * 16 * 256  # bytes of q_out


@pytest.mark.parametrize("over,msg", [
    (dict(pos=_words((3, 8), (1 << 20) + 32, ab.I32)), "q_out overlaps positions"),
    (dict(pos=_words((3, 8), (1 << 20) - 4, ab.I32)), "q_out overlaps positions"),
    (dict(pos=_words((3, 8), (1 << 20) + END - 4, ab.I32)), "q_out overlaps positions"),
    (dict(pos=_words((3, 8), (1 << 20) - 5000, ab.I32, [1000, 1])), "q_out overlaps positions"),  # its third axis
    (dict(pos=_words((3, 8), (3 << 19) + 64, ab.I32)), "k_out overlaps positions"),
    (dict(inv=_words((32,), (1 << 20) + 128, ab.F32)), "q_out overlaps inv_freq"),
    (dict(inv=_words((32,), (3 << 19) - 124, ab.F32)), "k_out overlaps inv_freq"),
    # in place: the inputs are outputs
    (dict(qo=ab._at((8, 16, 256), 0), pos=_words((3, 8), 256, ab.I32)), "q_out overlaps positions"),
])
def test_rope_refuses_outputs_over_positions_and_frequencies(over, msg):
    assert _rope(**over) == -1 and msg in pg.paged_gqa_last_error(), pg.paged_gqa_last_error()


@pytest.mark.gpu
def test_neighbours_of_the_outputs_are_no_overlap():
    """Positions and frequencies directly before and behind the outputs, in one allocation."""
    T, n = 8, 8 * 16 * 512
    buf = torch.zeros(4096 + n + 4096, dtype=torch.uint8, device="cuda")
    q = torch.randn(T, 16, 256).bfloat16().cuda()
    k, want, k_out = q[:, :2].clone(), torch.empty_like(q), torch.empty(T, 2, 256, dtype=torch.bfloat16, device="cuda")
    pos = torch.randint(0, 1000, (3, T), dtype=torch.int32).cuda()
    inv = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()
    pg.paged_gqa_rope(q, k, pos, inv, [16, 8, 8], want, k_out)
    out = buf[4096:4096 + n].view(torch.bfloat16).view(T, 16, 256)
    near = [buf[4096 - 96:4096].view(torch.int32).view(3, T), buf[4096 + n:4096 + n + 96].view(torch.int32).view(3, T)]
    for p in near:
        p.copy_(pos)
        pg.paged_gqa_rope(q, k, p, inv, [16, 8, 8], out, k_out)
        assert bool((out == want).all())
    f = buf[4096 + n:4096 + n + 128].view(torch.float32)
    f.copy_(inv)
    pg.paged_gqa_rope(q, k, pos, f, [16, 8, 8], out, k_out)
    assert bool((out == want).all())
