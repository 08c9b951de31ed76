"""Calls repeated many times give the same bits: a race between warps shows as a rare difference."""
import pytest
import torch

import paged_gqa_gb300 as pg
import workloads as wl
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,hkv", [("bf16", 1), ("bf16", 2), ("e4m3", 1)])
def test_a_split_batch_repeats_bit_for_bit(kv, hkv):
    """40 sequences of up to 40k keys, 1-4 new tokens, cut over all CTAs, under both planning paths."""
    gen = torch.Generator().manual_seed(605)
    Ls = torch.randint(1, 40000, (40,), generator=gen).tolist()
    qs = torch.randint(1, 5, (40,), generator=gen).tolist()
    spec = wl.CaseSpec("repeat", [(min(q, L), L) for q, L in zip(qs, Ls)], 16 * hkv, hkv, 16, kv_dtype=kv)
    case = wl.make_case(spec, device="cuda", seed=605, poison=True)
    first = gu.run_library(case)
    gu.check_full(case, first, f"{kv} caches, {hkv} kv heads")
    for i in range(150):
        prev = pg.paged_gqa_set_path(3 if i % 4 == 3 else 0)
        try:
            again = gu.run_library(case)
        finally:
            pg.paged_gqa_set_path(prev)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16)), f"call {i}"
