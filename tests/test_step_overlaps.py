"""Outputs of tree attention that share memory with what the call reads: host side, no GPU needed."""
import ctypes

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
