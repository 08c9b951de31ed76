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


def _cache(offset, shape=ab.CACHE, stride=None):
    return FakeTensor(shape, ab.U8, ptr=(1 << 26) + offset, stride=stride)


PAGE = 16 * 144          # of one head; CACHE has 2 heads
BOTH = [4 * PAGE, PAGE, 144, 1]          # the strides of one half of [pages, 2, heads, 16, 144]
INNER = [4 * PAGE, 2 * PAGE, 144, 1]     # and of [pages, heads, 2, 16, 144]


@pytest.mark.parametrize("k,v", [
    (_cache(0), _cache(16)),
    (_cache(0), _cache(9 * 2 * PAGE)),                       # k's last page is v's first
    (_cache(0, stride=BOTH), _cache(PAGE, stride=BOTH)),     # k's second head is v's first
    (_cache(0, stride=BOTH), _cache(2 * PAGE - 16, stride=BOTH)),
    (_cache(0, stride=BOTH), _cache(4 * PAGE, stride=BOTH)),  # v's pages are k's next ones
    (_cache(0, stride=INNER), _cache(2 * PAGE, stride=INNER)),
    (_cache(0, stride=INNER), _cache(PAGE, stride=BOTH)),    # the same page stride, other heads
])
def test_write_refuses_caches_that_overlap(k, v):
    for a, b in ((k, v), (v, k)):
        far = dict(k=a, v=b, kn=ab._at((8, 2, 256), 0), vn=ab._at((8, 2, 256), 1 << 20))
        assert ab._write(ab._args(**far)) == -1 and "k_cache and v_cache overlap" in pg.paged_gqa_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["[2, pages, heads]", "[pages, 2, heads]", "[pages, heads, 2]", "[heads, pages, 2]"])
def test_caches_of_one_allocation_are_no_overlap(layout):
    NB, H, P, T = 6, 2, 16, 40
    order = {"[2, pages, heads]": (2, NB, H), "[pages, 2, heads]": (NB, 2, H), "[pages, heads, 2]": (NB, H, 2),
             "[heads, pages, 2]": (H, NB, 2)}[layout]
    whole = torch.zeros(*order, P, 144, dtype=torch.uint8, device="cuda")
    axis = layout.strip("[]").split(", ").index("2")
    k, v = whole.select(axis, 0), whole.select(axis, 1)
    if layout.startswith("[heads"):
        k, v = k.transpose(0, 1), v.transpose(0, 1)
    kn, vn = (torch.randn(T, H, 256).bfloat16().cuda() for _ in range(2))
    table = torch.tensor([[3, 0, 5, 1]], dtype=torch.int32, device="cuda")
    lens, qsl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([50], [0, T]))
    pg.paged_gqa_cache_write_fp4(kn, vn, k, v, table, lens, qsl, 0.01, 0.02)
    want = [torch.zeros(NB, H, P, 144, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pg.paged_gqa_cache_write_fp4(kn, vn, *want, table, lens, qsl, 0.01, 0.02)
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()
    assert bool((k == want[0]).all()) and bool((v == want[1]).all())
