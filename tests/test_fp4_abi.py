"""Refusals of the 4-bit cache's and the rotary entry points: host side, no GPU needed."""
import ctypes

import pytest
import torch

import paged_gqa_gb300 as pg
from paged_gqa_gb300 import _binding as B
from tests.test_abi import FakeTensor

U8, BF, I32, F32 = torch.uint8, torch.bfloat16, torch.int32, torch.float32
CACHE = (10, 2, 16, 144)


def _desc(t):
    return B._desc(t, B.PG_FP4 if t.dtype is U8 and t.dim() == 4 else None)


def _args(**over):
    a = dict(q=FakeTensor((8, 16, 256), BF), kn=FakeTensor((8, 2, 256), BF), vn=FakeTensor((8, 2, 256), BF),
             k=FakeTensor(CACHE, U8), v=FakeTensor(CACHE, U8), bt=FakeTensor((2, 5), I32), sl=FakeTensor((2,), I32),
             qsl=FakeTensor((3,), I32), out=FakeTensor((8, 16, 256), BF))
    a.update(over)
    return a


def _attn(a, kd=1.0, vd=1.0, scale=1 / 16, ws=None):
    d = [_desc(a[n]) for n in ("q", "k", "v", "bt", "sl", "qsl", "out")]
    r = [ctypes.byref(x) for x in d]
    if ws is not None:
        return pg.load().paged_gqa_attn_fp4_ex(*r[:6], kd, vd, scale, r[6], *ws, None)
    return pg.load().paged_gqa_attn_fp4(*r[:6], kd, vd, scale, r[6], None)


def _write(a, kd=1.0, vd=1.0):
    d = [_desc(a[n]) for n in ("kn", "vn", "k", "v", "bt", "sl", "qsl")]
    return pg.load().paged_gqa_cache_write_fp4(*[ctypes.byref(x) for x in d], kd, vd, None)


def _read(a, kd=1.0, vd=1.0):
    d = [_desc(a[n]) for n in ("k", "v", "bt", "sl", "qsl", "kn", "vn")]
    r = [ctypes.byref(x) for x in d]
    return pg.load().paged_gqa_cache_read_fp4(*r[:5], kd, vd, *r[5:], None)


BAD_CACHES = [
    (dict(k=FakeTensor((10, 2, 16, 256), U8), v=FakeTensor((10, 2, 16, 256), U8)), -2, "144 bytes"),
    (dict(k=FakeTensor(CACHE, BF), v=FakeTensor(CACHE, BF)), -2, "4-bit"),
    (dict(v=FakeTensor((11, 2, 16, 144), U8)), -1, "shapes differ"),
    (dict(k=FakeTensor((10, 2, 24, 144), U8), v=FakeTensor((10, 2, 24, 144), U8)), -2, "page size"),
    (dict(k=FakeTensor(CACHE, U8, stride=[4608, 144, 288, 1])), -1, "contiguous"),
    (dict(v=FakeTensor(CACHE, U8, stride=[4616, 2304, 144, 1])), -1, "16 bytes"),
    (dict(v=FakeTensor(CACHE, U8, ptr=(1 << 20) + 8)), -1, "aligned"),
    (dict(bt=FakeTensor((3, 5), I32)), -1, "block_table rows"),
    (dict(qsl=FakeTensor((2,), I32)), -1, "query_start_loc"),
    (dict(sl=FakeTensor((2,), F32)), -1, "int32"),
    (dict(bt=FakeTensor((2, 5), I32, stride=[10, 2])), -1, "contiguous"),
    (dict(bt=FakeTensor((2, 5), I32, ptr=(1 << 20) + 2)), -1, "4-byte aligned"),
]


@pytest.mark.parametrize("over,code,msg", BAD_CACHES)
@pytest.mark.parametrize("call", [_attn, _write, _read])
def test_bad_caches_and_tables_are_refused(call, over, code, msg):
    assert call(_args(**over)) == code
    assert msg in pg.paged_gqa_last_error()


@pytest.mark.parametrize("over,code,msg", [
    (dict(q=FakeTensor((8, 16, 256), U8)), -2, "q must be bf16"),
    (dict(q=FakeTensor((8, 16, 128), BF)), -2, "head_dim"),
    (dict(q=FakeTensor((8, 15, 256), BF), out=FakeTensor((8, 15, 256), BF)), -1, "multiple"),
    (dict(q=FakeTensor((8, 16, 256), BF, stride=[4100, 256, 1])), -1, "16 bytes"),
    (dict(out=FakeTensor((9, 16, 256), BF)), -1, "out shape"),
    (dict(out=FakeTensor((8, 16, 256), F32)), -2, "out must be bf16"),
    (dict(out=FakeTensor((8, 16, 256), BF, stride=[0, 256, 1])), -1, "overlap"),
    (dict(k=FakeTensor((0, 2, 16, 144), U8), v=FakeTensor((0, 2, 16, 144), U8)), -1, "without pages"),
    (dict(bt=FakeTensor((2, 0), I32)), -1, "without pages"),
])
def test_attention_refusals(over, code, msg):
    assert _attn(_args(**over)) == code
    assert msg in pg.paged_gqa_last_error()


def test_attention_refuses_scales_that_do_not_fit():
    for kw in (dict(kd=float("nan")), dict(vd=float("inf")), dict(scale=float("inf")), dict(kd=3e38, scale=1e3)):
        assert _attn(_args(), **kw) == -1


def test_write_and_read_refusals():
    assert _write(_args(kn=FakeTensor((8, 2, 256), U8))) == -2
    assert _write(_args(kn=FakeTensor((8, 3, 256), BF), vn=FakeTensor((8, 3, 256), BF))) == -1
    assert "num_kv_heads" in pg.paged_gqa_last_error()
    assert _write(_args(vn=FakeTensor((7, 2, 256), BF))) == -1
    assert _read(_args(kn=FakeTensor((8, 2, 256), BF, stride=[256, 256, 1]))) == -1
    assert "overlap" in pg.paged_gqa_last_error()
    # written pages that overlap; a read of them is fine, so only the write refuses
    assert _write(_args(k=FakeTensor(CACHE, U8, stride=[4608, 2288, 144, 1]))) == -1
    assert "overlap" in pg.paged_gqa_last_error()
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert _write(_args(), kd=bad) == -1 and _read(_args(), vd=bad) == -1
        assert "descales" in pg.paged_gqa_last_error()
    none = dict(bt=FakeTensor((0, 5), I32), sl=FakeTensor((0,), I32), qsl=FakeTensor((1,), I32))
    assert _write(_args(**none)) == -1
    assert "without sequences" in pg.paged_gqa_last_error()


def test_empty_batches_are_no_ops():
    none = dict(bt=FakeTensor((0, 5), I32), sl=FakeTensor((0,), I32), qsl=FakeTensor((1,), I32),
                q=FakeTensor((0, 16, 256), BF), out=FakeTensor((0, 16, 256), BF), kn=FakeTensor((0, 2, 256), BF),
                vn=FakeTensor((0, 2, 256), BF))
    assert _attn(_args(**none)) == 0 and _write(_args(**none)) == 0 and _read(_args(**none)) == 0
    assert _attn(_args(**none), ws=(None, 0)) == 0


def _rope(sections=(16, 8, 8), interleaved=0, adjacent=0, n_axes=None, **over):
    a = dict(q=FakeTensor((8, 16, 256), BF), k=FakeTensor((8, 2, 256), BF), pos=FakeTensor((3, 8), I32),
             inv=FakeTensor((32,), F32), qo=FakeTensor((8, 16, 256), BF, ptr=1 << 24),
             ko=FakeTensor((8, 2, 256), BF, ptr=1 << 25))
    a.update(over)
    d = [B._desc(a[n]) for n in ("q", "k", "pos", "inv", "qo", "ko")]
    r = [ctypes.byref(x) for x in d]
    s = None if sections is None else (ctypes.c_int32 * len(sections))(*sections)
    return pg.load().paged_gqa_rope(*r[:4], s, interleaved, adjacent, *r[4:], None)


@pytest.mark.parametrize("over,code,msg", [
    (dict(q=FakeTensor((8, 16, 256), F32)), -2, "q must be bf16"),
    (dict(k=FakeTensor((8, 2, 128), BF)), -2, "head_dim"),
    (dict(k=FakeTensor((7, 2, 256), BF), ko=FakeTensor((7, 2, 256), BF, ptr=1 << 25)), -1, "number of tokens"),
    (dict(qo=FakeTensor((8, 15, 256), BF)), -1, "q_out shape"),
    (dict(qo=FakeTensor((8, 16, 256), BF, stride=[8192, 256, 1], ptr=1 << 20)), -1, "same strides"),
    (dict(ko=FakeTensor((8, 2, 256), BF, stride=[256, 128, 1], ptr=1 << 25)), -1, "overlap"),
    (dict(pos=FakeTensor((3, 8), torch.bfloat16)), -1, "int32"),
    (dict(pos=FakeTensor((5, 8), I32)), -2, "axes"),
    (dict(pos=FakeTensor((3, 9), I32)), -1, "[axes, T]"),
    (dict(pos=FakeTensor((3, 8), I32, stride=[16, 2])), -1, "contiguous"),
    (dict(inv=FakeTensor((32,), torch.bfloat16)), -1, "float32"),
    (dict(inv=FakeTensor((136,), F32)), -2, "8 to 128"),
    (dict(inv=FakeTensor((12,), F32)), -2, "multiple of 8"),
    (dict(sections=(16, 8, 7)), -1, "add up"),
    (dict(sections=(40, -4, -4)), -1, "negative"),
    (dict(sections=None), -1, "null sections"),
    (dict(sections=(10, 11, 11), interleaved=1), -1, "no 11-th"),
])
def test_rope_refusals(over, code, msg):
    assert _rope(**over) == code
    assert msg in pg.paged_gqa_last_error()


def test_rope_without_tokens_is_a_no_op():
    assert _rope(q=FakeTensor((0, 16, 256), BF), k=FakeTensor((0, 2, 256), BF), pos=FakeTensor((3, 0), I32),
                 qo=FakeTensor((0, 16, 256), BF, ptr=1 << 24), ko=FakeTensor((0, 2, 256), BF, ptr=1 << 25)) == 0


def test_python_calls_refuse_host_tensors_and_other_types():
    if not torch.cuda.is_available():
        # the device check itself needs a CUDA build's current device
        pytest.skip("no CUDA device")
    q = torch.zeros(1, 16, 256, dtype=BF)
    with pytest.raises(ValueError, match="current CUDA device"):
        pg.paged_gqa_rope(q, q, torch.zeros(1, 1, dtype=I32), torch.zeros(8), [8])


def test_marshalling_refuses_caches_of_another_type():
    k = FakeTensor(CACHE, torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="uint8"):
        B._pack_fp4(0, k, k)


def _at(shape, offset, stride=None):
    return FakeTensor(shape, BF, ptr=(1 << 24) + 2 * offset, stride=stride)


ROW = 20 * 256  # a token of a projection's output: 16 query heads, 2 key heads, 2 value heads


@pytest.mark.parametrize("over,msg", [
    # q_out where k is; q_out half over q; the outputs at one place; a token apart
    (dict(q=_at((8, 2, 256), 0), k=_at((8, 2, 256), 1 << 20), qo=_at((8, 2, 256), 1 << 20), ko=_at((8, 2, 256), 1 << 21)), "q_out overlaps k"),
    (dict(q=_at((8, 16, 256), 0), qo=_at((8, 16, 256), 8 * 256)), "q_out overlaps q without"),
    (dict(k=_at((8, 2, 256), 1 << 20), ko=_at((8, 2, 256), (1 << 20) + 3 * 512)), "k_out overlaps k without"),
    (dict(qo=_at((8, 16, 256), 1 << 20), ko=_at((8, 2, 256), (1 << 20) + 7 * 16 * 256)), "q_out overlaps k_out"),
    (dict(q=_at((8, 16, 256), 0, [ROW, 256, 1]), qo=_at((8, 16, 256), 0, [ROW, 256, 1]),
          k=_at((8, 2, 256), 15 * 256, [ROW, 256, 1]), ko=_at((8, 2, 256), 1 << 20)), "q_out overlaps k"),
    (dict(q=_at((8, 16, 256), 0, [ROW, 256, 1]), qo=_at((8, 16, 256), 0, [ROW, 256, 1]),
          k=_at((8, 2, 256), 1 << 20), ko=_at((8, 2, 256), 5 * ROW + 17 * 256 - 3 * ROW - 2 * 256, [ROW, 256, 1])), "k_out overlaps q"),
])
def test_rope_refuses_overlapping_tensors(over, msg):
    a = dict(q=_at((8, 16, 256), 0), k=_at((8, 2, 256), 1 << 18), qo=_at((8, 16, 256), 1 << 19), ko=_at((8, 2, 256), 3 << 18))
    a.update(over)
    assert _rope(**a) == -1 and msg in pg.paged_gqa_last_error(), pg.paged_gqa_last_error()


def test_write_and_read_refuse_one_memory_for_two_tensors():
    far = dict(k=FakeTensor(CACHE, U8, ptr=1 << 22), kn=_at((8, 2, 256), 0), vn=_at((8, 2, 256), 1 << 20))
    assert _write(_args(**dict(far, v=FakeTensor(CACHE, U8, ptr=1 << 22)))) == -1 and "same memory" in pg.paged_gqa_last_error()
    assert _read(_args(**dict(far, vn=_at((8, 2, 256), 256)))) == -1 and "k_out and v_out overlap" in pg.paged_gqa_last_error()


def test_attention_refuses_an_output_over_its_queries():
    assert _attn(_args(q=_at((8, 16, 256), 0), out=_at((8, 16, 256), 256 * 16))) == -1
    assert "out overlaps q" in pg.paged_gqa_last_error()
