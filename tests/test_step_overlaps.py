"""Outputs of tree attention and caches of keep that share memory with what the call reads: host side, no GPU needed."""
import ctypes
import itertools
import random

import pytest
import torch

import paged_gqa_gb300 as pg
from paged_gqa_gb300 import _binding as B
from tests.test_abi import FakeTensor

U8, BF, I32 = torch.uint8, torch.bfloat16, torch.int32
OUT = 1 << 30


def _tree(out=None, **over):
    a = dict(q=FakeTensor((8, 16, 256), BF, ptr=1 << 24), k=FakeTensor((10, 16, 2, 256), U8, ptr=2 << 24),
             v=FakeTensor((10, 16, 2, 256), U8, ptr=3 << 24), bt=FakeTensor((2, 5), I32, ptr=4 << 24), lens=FakeTensor((2,), I32, ptr=5 << 24),
             qsl=FakeTensor((3,), I32, ptr=6 << 24), masks=FakeTensor((8, 1), I32, ptr=7 << 24), out=out or FakeTensor((8, 16, 256), BF, ptr=OUT))
    a.update(over)
    r = [ctypes.byref(B._desc(x)) for x in a.values()]
    code = pg.load().paged_gqa_attn_tree(*r[:7], 1.0, 1.0, 1 / 16, r[7], None)
    return code, pg.paged_gqa_last_error()


@pytest.mark.parametrize("name,arg,shape", [("masks", "masks", (8, 1)), ("block_table", "bt", (2, 5)), ("seq_lens", "lens", (2,)),
                                            ("query_start_loc", "qsl", (3,))])
def test_out_over_what_tree_attention_reads_is_refused(name, arg, shape):
    end = OUT + 8 * 16 * 512
    n = 4 * torch.Size(shape).numel()
    for at in (OUT, OUT + 512, end - 4, OUT - n + 4, end - n):
        code, msg = _tree(**{arg: FakeTensor(shape, I32, ptr=at)})
        assert code == -1 and msg == f"out overlaps {name}", at
    for at in (OUT - n, end):  # right in front of it and behind it
        assert "overlaps" not in _tree(**{arg: FakeTensor(shape, I32, ptr=at)})[1]


def test_what_lies_between_the_rows_of_out():
    """Each token's rows of out with 16 bytes behind them: what lies there wholly is told apart, a tensor that steps over
    rows of out is not."""
    out = FakeTensor((8, 16, 256), BF, ptr=OUT, stride=[16 * 256 + 8, 256, 1])
    one = FakeTensor((2,), I32, ptr=OUT + 16 * 512 + 8)
    assert "overlaps" not in _tree(out=out, lens=one)[1]
    assert _tree(out=out, lens=FakeTensor((2,), I32, ptr=OUT + 16 * 512 + 12))[1] == "out overlaps seq_lens"
    assert _tree(out=out, masks=FakeTensor((8, 1), I32, ptr=OUT + 16 * 512, stride=[4, 1]))[1] == "out overlaps masks"
    assert "overlaps" not in _tree(masks=FakeTensor((8, 1), I32, ptr=OUT - 4, stride=[-4, 1]))[1]


KEEP = dict(bt=(2, 5), lens=(2,), qsl=(3,), kept=(2, 4), num=(2,), lens_out=(2,))
NAMES = dict(bt="block_table", lens="seq_lens", qsl="query_start_loc", kept="kept", num="num_kept", lens_out="seq_lens_out")


def _keep(k, v, **at):
    a = dict(k=k, v=v)
    for i, (name, shape) in enumerate(KEEP.items()):
        a[name] = FakeTensor(shape, I32, ptr=at.get(name, (i + 1) << 24))
    code = pg.load().paged_gqa_cache_keep(*[ctypes.byref(B._desc(x)) for x in a.values()], None)
    return code, pg.paged_gqa_last_error()


@pytest.mark.parametrize("name", list(KEEP))
@pytest.mark.parametrize("dtype", [U8, BF])
def test_integers_in_a_cache_are_refused_by_keep(name, dtype):
    size = 10 * 16 * 2 * 256 * (2 if dtype is BF else 1)
    n = 4 * torch.Size(KEEP[name]).numel()
    k, v = FakeTensor((10, 16, 2, 256), dtype, ptr=1 << 30), FakeTensor((10, 16, 2, 256), dtype, ptr=2 << 30)
    for base, cache in ((1 << 30, "k_cache"), (2 << 30, "v_cache")):
        for at in (base, base - n + 4, base + size - 4, base + size // 2):
            assert _keep(k, v, **{name: at}) == (-1, f"{NAMES[name]} overlaps {cache}")
        for at in (base - n, base + size):
            assert "overlaps" not in _keep(k, v, **{name: at})[1]


def test_integers_between_the_rows_of_a_cache():
    """Every order of the dims and gaps behind the rows of each: a cache's rows are told from what lies between them exactly."""
    r = random.Random(2)
    shape, base, seen = (3, 16, 2), 1 << 30, [0, 0]
    far = FakeTensor((3, 16, 2, 256), U8, ptr=3 << 30)
    for order in itertools.permutations(range(3)):
        for gaps in itertools.product((0, 32, 256), repeat=3):
            strides, at = [0, 0, 0], 256 + gaps[0]
            for d, gap in zip(reversed(order), (*gaps[1:], 0)):
                strides[d] = at
                at = at * shape[d] + gap
            rows = [base + sum(c * s for c, s in zip(i, strides)) for i in itertools.product(*map(range, shape))]
            k = FakeTensor((*shape, 256), U8, ptr=base, stride=strides + [1])
            for _ in range(12):
                x = r.choice(rows) + r.choice([-8, -4, 0, 252, 256, 260, 256 + gaps[0] - 8, 256 + gaps[0] - 4, 4 * r.randrange(-64, 128)])
                want = any(x < y + 256 and y < x + 8 for y in rows)
                assert ("overlaps" in _keep(k, far, lens=x)[1]) == want, (strides, x - base)
                seen[want] += 1
    assert min(seen) > 100
