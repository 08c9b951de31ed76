"""4-bit attention repeated many times gives the same bits (a race between warps shows as a rare difference),
and long split rows are right each by its own size."""
import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import fp4_util as fu

pytestmark = pytest.mark.gpu

DECODE, VERIFY, PREFILL = 128, 2, 4


def _ragged(n, q_hi, seed, l_hi=40000):
    gen = torch.Generator().manual_seed(seed)
    Ls = torch.randint(1, l_hi, (n,), generator=gen).tolist()
    qs = torch.randint(1, q_hi + 1, (n,), generator=gen).tolist()
    return [(min(q, L), L) for q, L in zip(qs, Ls)]


def _run(c):
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pg.paged_gqa_attn_fp4(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out)
    return out


# name, sequences, q heads, kv heads, the kernels that serve it
SPLIT = [
    ("single tokens", _ragged(40, 1, 1), 8, 1, DECODE),
    ("single tokens, two kv heads", _ragged(23, 1, 2), 12, 2, DECODE),
    ("verify", _ragged(40, 4, 3), 16, 1, VERIFY),
    ("verify, two kv heads", _ragged(30, 4, 4), 32, 2, VERIFY),
    ("prefill", [(130, 9000), (311, 400), (77, 20000), (600, 600)], 8, 1, PREFILL),
    ("mixed", _ragged(9, 4, 5, 9000) + [(150, 7000), (290, 3000)], 24, 2, VERIFY | PREFILL),
]


@pytest.mark.parametrize("i", range(len(SPLIT)), ids=[s[0] for s in SPLIT])
def test_a_split_batch_repeats_bit_for_bit(i):
    name, seqs, hq, hkv, bits = SPLIT[i]
    c = fu.make(seqs, hq, hkv, 16, seed=400 + i)
    first = _run(c)
    assert pg.paged_gqa_last_plan()["path_bits"] & bits == bits
    assert bool(first.isfinite().all())
    for n in range(150):
        prev = pg.paged_gqa_set_path(3 if n % 4 == 3 else 0)
        try:
            again = _run(c)
        finally:
            pg.paged_gqa_set_path(prev)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16)), f"call {n}"
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()


# (few rows: the 64-bit reference walks every key of each)
LONG = [
    ("single tokens", [(1, 30000), (1, 7777), (1, 16), (1, 17)], 8, 1, DECODE),
    ("verify", [(4, 30000), (2, 12345), (1, 9), (3, 31)], 16, 1, VERIFY),
    ("verify, two kv heads", [(2, 20000), (1, 40), (4, 5000)], 16, 2, VERIFY),
    ("prefill", [(20, 20000), (9, 9), (70, 100)], 16, 1, PREFILL),
]


@pytest.mark.parametrize("path", [0, 2, 3])
@pytest.mark.parametrize("i", range(len(LONG)), ids=[s[0] for s in LONG])
def test_each_row_of_a_long_split_sequence(i, path):
    """Per row, the relative L2 over its 256 values. The output's rounding to bf16 and P's to f16 are off by
    2^-8 and 2^-11 of a value at most, a split piece's f16 partial by 2^-11 of one; P's errors do not follow
    V's signs, so that over n equal weights they meet as 2^-11 / sqrt(n) of |V| where the output is
    |V| / sqrt(n): as relative errors they add as they are. 2^-8 + 3 * 2^-11 = 5.4e-3; a row that lost
    one of 30 pieces is off by about 18 %."""
    name, seqs, hq, hkv, bits = LONG[i]
    c = fu.make(seqs, hq, hkv, 32, seed=420 + i)
    prev = pg.paged_gqa_set_path(path)
    try:
        out = _run(c)
        if path != 2:
            assert pg.paged_gqa_last_plan()["path_bits"] & bits == bits
    finally:
        pg.paged_gqa_set_path(prev)
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()
    rows = np.arange(c.T * hq)
    ref = fu.reference(c, rows).reshape(len(rows), fu.D)
    got = out.double().cpu().numpy().reshape(-1, fu.D)
    rel = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert (rel <= 2.0 ** -8 + 3 * 2.0 ** -11).all(), f"{name}: row {rel.argmax()} is off by {rel.max():.3g}"
