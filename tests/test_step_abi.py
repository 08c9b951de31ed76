"""Refusals of the block table, token tree and prompt entry points: host side, no GPU needed."""
import ctypes

import pytest
import torch

import paged_gqa_gb300 as pg
from paged_gqa_gb300 import _binding as B
from tests.test_abi import FakeTensor

U8, BF, F16, I32, F32 = torch.uint8, torch.bfloat16, torch.float16, torch.int32, torch.float32


def ints(*shape, at=1, **kw):
    return FakeTensor(shape, I32, ptr=at << 24, **kw)


def _refs(a):
    return [ctypes.byref(B._desc(x)) for x in a.values()]


def _same(a, over):
    assert set(over) <= set(a), over
    a.update(over)
    return a


def _tables(page=16, **over):
    a = _same(dict(q=ints(4), ctx=ints(4, at=2), rows=ints(4, at=3), pages=ints(9, 20, at=4), counts=ints(9, at=5), free=ints(50, at=6),
                   num=ints(1, at=7), table=ints(4, 20, at=8), lens=ints(4, at=9), qsl=ints(5, at=10), slots=ints(7, at=11),
                   counts_out=ints(9, at=12), num_out=ints(1, at=13)), over)
    r = _refs(a)
    return pg.load().paged_gqa_build_tables(*r[:3], page, *r[3:], None)


@pytest.mark.parametrize("over,code,msg", [
    (dict(q=ints(5)), -1, "must match q_lens"),
    (dict(rows=FakeTensor((4,), F32)), -1, "int32"),
    (dict(qsl=ints(4, at=10)), -1, "must match q_lens"),
    (dict(table=ints(4, 20, at=8, stride=[20, 2])), -1, "contiguous"),
    (dict(table=ints(4, 20, at=8, stride=[19, 1])), -1, "rows overlap"),
    (dict(pages=ints(9, 20, at=4, stride=[0, 1])), -1, "rows overlap"),
    (dict(counts=ints(8, at=5)), -1, "entry per row"),
    (dict(counts_out=ints(8, at=12)), -1, "entry per row"),
    (dict(num=ints(2, at=7)), -1, "one entry"),
    (dict(slots=FakeTensor((7,), I32, ptr=(11 << 24) + 2)), -1, "4-byte aligned"),
    (dict(lens=ints(4, at=1)), -1, "seq_lens overlaps q_lens"),
    (dict(lens=FakeTensor((4,), I32, ptr=(10 << 24) + 16)), -1, "seq_lens overlaps query_start_loc"),
    (dict(free=FakeTensor((50,), I32, ptr=(4 << 24) + 700)), -1, "pages overlaps free_pages"),
    (dict(counts_out=FakeTensor((9,), I32, ptr=(5 << 24) + 4)), -1, "page_counts_out overlaps page_counts"),
    (dict(q=ints(4, 1)), -1, "expected 1 dims"),
    (dict(slots=FakeTensor((7,), I32, ptr=0)), -1, "null"),
    (dict(q=ints(8193), ctx=ints(8193, at=2), rows=ints(8193, at=3), table=ints(8193, 20, at=8), lens=ints(8193, at=9), qsl=ints(8194, at=10)),
     -2, "8192 requests"),
])
def test_table_refusals(over, code, msg):
    assert _tables(**over) == code
    assert msg in pg.paged_gqa_last_error()


def test_table_page_sizes():
    for page in (0, -16, 8, 24, 256):
        assert _tables(page=page) == -2 and "page size" in pg.paged_gqa_last_error()


def _masks(**over):
    a = _same(dict(parents=ints(9), lens=ints(2, at=2), qsl=ints(3, at=3), masks=ints(9, 2, at=4), positions=ints(3, 9, at=5)), over)
    return pg.load().paged_gqa_tree_masks(*_refs(a), None)


@pytest.mark.parametrize("over,code,msg", [
    (dict(parents=FakeTensor((9,), F32)), -1, "int32"),
    (dict(lens=ints(3, at=2)), -1, "length must match"),
    (dict(masks=ints(8, 2, at=4)), -1, "[T, words]"),
    (dict(masks=ints(9, 0, at=4)), -2, "words"),
    (dict(masks=ints(9, 33, at=4)), -2, "words"),
    (dict(masks=ints(9, 2, at=4, stride=[1, 1])), -1, "rows overlap"),
    (dict(positions=ints(3, 8, at=5)), -1, "[axes, T]"),
    (dict(positions=ints(5, 9, at=5)), -2, "axes"),
    (dict(positions=ints(3, 9, at=4)), -1, "masks overlaps positions"),
    (dict(parents=ints(9, at=5)), -1, "positions overlaps parents"),
])
def test_mask_refusals(over, code, msg):
    assert _masks(**over) == code
    assert msg in pg.paged_gqa_last_error()


def _tree(kd=1.0, vd=1.0, scale=1 / 16, ws=None, **over):
    a = _same(dict(q=FakeTensor((8, 16, 256), BF), k=FakeTensor((10, 16, 2, 256), U8), v=FakeTensor((10, 16, 2, 256), U8),
                   bt=ints(2, 5), lens=ints(2), qsl=ints(3), masks=ints(8, 1), out=FakeTensor((8, 16, 256), BF, ptr=1 << 30)), over)
    r = _refs(a)
    if ws is not None:
        return pg.load().paged_gqa_attn_tree_ex(*r[:7], kd, vd, scale, r[7], *ws, None)
    return pg.load().paged_gqa_attn_tree(*r[:7], kd, vd, scale, r[7], None)


@pytest.mark.parametrize("over,code,msg", [
    (dict(q=FakeTensor((8, 16, 256), U8)), -2, "bf16 q"),
    (dict(q=FakeTensor((8, 15, 256), BF), out=FakeTensor((8, 15, 256), BF, ptr=1 << 30)), -1, "multiple"),
    (dict(k=FakeTensor((10, 24, 2, 256), U8), v=FakeTensor((10, 24, 2, 256), U8)), -2, "page size"),
    (dict(masks=FakeTensor((8, 1), F32)), -1, "int32"),
    (dict(masks=ints(7, 1)), -1, "[T, words]"),
    (dict(masks=ints(8, 33)), -2, "words"),
    (dict(masks=ints(8, 0)), -2, "words"),
    (dict(masks=ints(8, 2, stride=[2, 2])), -1, "contiguous"),
    (dict(masks=FakeTensor((8, 1), I32, ptr=0)), -1, "null"),
    (dict(bt=FakeTensor((2, 5), I32, ptr=(1 << 20) + 2)), -1, "4-byte aligned"),
    (dict(out=FakeTensor((8, 16, 256), BF)), -1, "out overlaps q"),
    (dict(bt=ints(2, 0)), -1, "without pages"),
    (dict(kd=3e38, scale=1e9), -1, "fit fp32"),
    (dict(vd=float("nan")), -1, "finite"),
])
def test_tree_refusals(over, code, msg):
    assert _tree(**over) == code
    assert msg in pg.paged_gqa_last_error()


def _keep(**over):
    a = _same(dict(k=FakeTensor((10, 16, 2, 256), U8), v=FakeTensor((10, 16, 2, 256), U8, ptr=1 << 30), bt=ints(2, 5), lens=ints(2, at=2),
                   qsl=ints(3, at=3), kept=ints(2, 4, at=4), num=ints(2, at=5), lens_out=ints(2, at=6)), over)
    return pg.load().paged_gqa_cache_keep(*_refs(a), None)


@pytest.mark.parametrize("over,code,msg", [
    (dict(k=FakeTensor((10, 16, 2, 256), F16), v=FakeTensor((10, 16, 2, 256), F16, ptr=1 << 30)), -2, "dtype"),
    (dict(v=FakeTensor((10, 16, 2, 256), BF, ptr=1 << 30)), -1, "dtypes differ"),
    (dict(v=FakeTensor((11, 16, 2, 256), U8, ptr=1 << 30)), -1, "shapes differ"),
    (dict(k=FakeTensor((10, 16, 2, 128), U8), v=FakeTensor((10, 16, 2, 128), U8, ptr=1 << 30)), -2, "head_dim"),
    (dict(k=FakeTensor((10, 20, 2, 256), U8), v=FakeTensor((10, 20, 2, 256), U8, ptr=1 << 30)), -2, "page size"),
    (dict(k=FakeTensor((10, 16, 2, 256), U8, stride=[8192, 512, 0, 1])), -1, "overlap"),
    (dict(k=FakeTensor((10, 16, 2, 256), U8, stride=[8200, 512, 256, 1])), -1, "16 bytes"),
    (dict(v=FakeTensor((10, 16, 2, 256), U8, ptr=1 << 20)), -1, "k_cache and v_cache overlap"),
    (dict(kept=ints(3, 4, at=4)), -1, "must match seq_lens"),
    (dict(num=ints(3, at=5)), -1, "must match seq_lens"),
    (dict(lens_out=ints(2, at=2)), -1, "seq_lens_out overlaps seq_lens"),
    (dict(lens_out=FakeTensor((2,), I32, ptr=(4 << 24) + 28)), -1, "seq_lens_out overlaps kept"),
])
def test_keep_refusals(over, code, msg):
    assert _keep(**over) == code
    assert msg in pg.paged_gqa_last_error()


def _prompt(scale=1 / 16, **over):
    a = _same(dict(q=FakeTensor((9, 8, 256), BF), k=FakeTensor((9, 2, 256), BF, ptr=2 << 24), v=FakeTensor((9, 2, 256), BF, ptr=3 << 24),
                   qsl=ints(3, at=4), out=FakeTensor((9, 8, 256), BF, ptr=5 << 24), lse=FakeTensor((9, 8), F32, ptr=6 << 24)), over)
    lse = a.pop("lse")
    r = _refs(a)
    return pg.load().paged_gqa_attn_prompt(*r[:4], scale, r[4], ctypes.byref(B._desc(lse)) if lse is not None else None, None)


@pytest.mark.parametrize("over,code,msg", [
    (dict(q=FakeTensor((9, 8, 256), U8)), -2, "bf16 or f16"),
    (dict(k=FakeTensor((9, 2, 256), F16, ptr=2 << 24)), -2, "k must be bf16"),
    (dict(q=FakeTensor((9, 8, 256), F16)), -2, "must be f16"),
    (dict(k=FakeTensor((8, 2, 256), BF, ptr=2 << 24)), -1, "num_kv_heads"),
    (dict(v=FakeTensor((9, 1, 256), BF, ptr=3 << 24)), -1, "num_kv_heads"),
    (dict(k=FakeTensor((9, 3, 256), BF, ptr=2 << 24), v=FakeTensor((9, 3, 256), BF, ptr=3 << 24)), -1, "multiple"),
    (dict(q=FakeTensor((9, 258, 256), BF), out=FakeTensor((9, 258, 256), BF, ptr=5 << 26)), -2, "128 q heads"),
    (dict(out=FakeTensor((9, 8, 256), BF, ptr=2 << 24)), -1, "out overlaps k"),
    (dict(out=FakeTensor((9, 8, 256), BF, ptr=5 << 24, stride=[2048, 128, 1])), -1, "overlap"),
    (dict(q=FakeTensor((9, 8, 256), BF, stride=[2052, 256, 1])), -1, "16 bytes"),
    (dict(q=FakeTensor((9, 8, 256), BF, ptr=(1 << 20) + 8)), -1, "aligned"),
    (dict(qsl=FakeTensor((3,), F32, ptr=4 << 24)), -1, "int32"),
    (dict(qsl=ints(0, at=4)), -1, "query_start_loc"),
    (dict(qsl=FakeTensor((3,), I32, ptr=5 << 24)), -1, "out overlaps query_start_loc"),
    (dict(lse=FakeTensor((9, 8), BF, ptr=6 << 24)), -1, "float32"),
    (dict(lse=FakeTensor((8, 9), F32, ptr=6 << 24)), -1, "num_q_heads"),
    (dict(lse=FakeTensor((9, 8), F32, ptr=6 << 24, stride=[0, 1])), -1, "overlap"),
    (dict(lse=FakeTensor((9, 8), F32, ptr=5 << 24)), -1, "lse overlaps out"),
    (dict(lse=FakeTensor((9, 8), F32, ptr=3 << 24)), -1, "lse overlaps v"),
    (dict(scale=float("nan")), -1, "finite"),
    (dict(scale=3e38), -1, "finite"),
])
def test_prompt_refusals(over, code, msg):
    assert _prompt(**over) == code
    assert msg in pg.paged_gqa_last_error()


def test_empty_batches_are_no_ops():
    z, one = ints(0), ints(1)
    assert _masks(parents=z, lens=z, qsl=one, masks=ints(0, 1), positions=ints(1, 0)) == 0
    q = FakeTensor((0, 16, 256), BF)
    assert _tree(q=q, out=q, masks=ints(0, 1), bt=ints(0, 5), lens=z, qsl=one) == 0
    assert _tree(q=q, out=q, masks=ints(0, 1), bt=ints(0, 5), lens=z, qsl=one, ws=(None, 0)) == 0
    assert _keep(bt=ints(0, 5), lens=z, qsl=one, kept=ints(0, 3), num=z, lens_out=z) == 0
    kv = FakeTensor((0, 2, 256), BF)
    assert _prompt(q=FakeTensor((0, 8, 256), BF), k=kv, v=kv, qsl=one, out=FakeTensor((0, 8, 256), BF), lse=None) == 0


def _row_starts(ptr, strides, shape):
    return {ptr + b * strides[0] + p * strides[1] + h * strides[2] for b in range(shape[0]) for p in range(shape[1]) for h in range(shape[2])}


def test_keep_tells_interleaved_caches_from_overlapping_ones():
    import itertools
    import random
    r = random.Random(1)
    shape, base, seen = (3, 16, 2), 1 << 20, [0, 0]
    for order in itertools.permutations(range(3)):  # which dim is outermost
        for gap in (0, 256):
            strides, at = [0, 0, 0], 256 + gap
            for d in reversed(order):
                strides[d] = at
                at = at * shape[d] + r.choice([0, 256 + gap])
            for delta in [256, 512, 16, strides[0], strides[1], strides[2], strides[1] - 256, at, at + 16, at - 256] + [
                    16 * r.randrange(0, at // 16) for _ in range(12)]:
                a, b = _row_starts(base, strides, shape), _row_starts(base + delta, strides, shape)
                every = sorted([(x, 0) for x in a] + [(x, 1) for x in b])
                want = any(y[0] - x[0] < 256 and x[1] != y[1] for x, y in zip(every, every[1:]))
                st = strides + [1]
                _keep(k=FakeTensor((*shape, 256), U8, ptr=base, stride=st), v=FakeTensor((*shape, 256), U8, ptr=base + delta, stride=st))
                assert ("k_cache and v_cache overlap" in pg.paged_gqa_last_error()) == want, (order, gap, delta)
                seen[want] += 1
    assert min(seen) > 20


def test_keep_refuses_caches_of_unequal_strides_in_one_range():
    st = [8192 * 2, 512, 256, 1]
    assert _keep(k=FakeTensor((10, 16, 2, 256), U8, ptr=1 << 20, stride=st),
                 v=FakeTensor((10, 16, 2, 256), U8, ptr=(1 << 20) + 8192, stride=[8192 * 2, 256, 4096, 1])) == -1
    assert "k_cache and v_cache overlap" in pg.paged_gqa_last_error()
