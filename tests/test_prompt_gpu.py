"""Attention over whole packed prompts, against the definition in 64 bits."""
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import step_util as su

pytestmark = pytest.mark.gpu

SMALL = [
    ([1], 1, 1), ([2, 1, 0, 3], 8, 1), ([173], 8, 1), ([128, 129, 127, 1, 64], 4, 2), ([300, 7, 95], 16, 2), ([33, 700], 24, 2), ([260, 1], 3, 1),
    ([100, 31], 6, 1), ([65, 64, 63], 5, 5), ([1] * 90, 12, 1), ([513], 128, 1), ([40, 41], 100, 1), ([1100], 2, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(SMALL)))
@pytest.mark.parametrize("path", [0, 1])
def test_prompts(path, case, dtype):
    lens, hq, hkv = SMALL[case]
    x = su.Prompt(lens, hq, hkv, dtype, seed=case, fused=case % 2 == 0)
    prev = pg.paged_gqa_set_path(path)
    try:
        out, lse = x.run()
    finally:
        pg.paged_gqa_set_path(prev)
    x.check(out, lse)


def test_longer_prompts():
    x = su.Prompt([2500, 1, 1777], 8, 1, seed=3)
    out, lse = x.run()
    x.check(out, lse, rows={0: [0, 1, 127, 128, 129, 1000, 2047, 2499], 1: [0], 2: [0, 255, 256, 1776]})
    same, _ = x.run(lse=False)
    assert torch.equal(out, same)


@pytest.mark.parametrize("scale", [-1 / 16, 0.0, 1.0, 3.0])
def test_scales(scale):
    x = su.Prompt([200, 45], 8, 2, seed=5, scale=scale)
    out, lse = x.run()
    x.check(out, lse)


def test_rows_of_no_prompt_stay():
    x = su.Prompt([150, 20], 8, 1, seed=7, behind=40)
    out, lse = x.run(out=torch.full((210, 8, 256), 5.0, dtype=torch.bfloat16, device="cuda"))
    assert (out[170:] == 5).all() and torch.isnan(lse[170:]).all()
    x.check(out, lse)


def test_nan_in_one_prompt_reaches_no_other():
    x = su.Prompt([100, 150, 64], 8, 2, seed=8)
    for t in (x.q, x.k, x.v):
        t[100:250] = float("nan")
    out, lse = x.run()
    assert torch.isnan(out[100:250]).all()
    x.check(out, lse, rows={0: list(range(100)), 2: list(range(64))})


def test_bad_starts_are_flagged():
    x = su.Prompt([50, 60], 8, 1)
    x.qsl_t = torch.tensor([0, 50, 111], dtype=torch.int32, device="cuda")
    out, _ = x.run(check=False)
    assert pg.paged_gqa_check_device_errors() == -5
    assert torch.isnan(out[50:]).all()
    x.check(out, None, rows={0: list(range(50))})
    x.qsl_t = torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")
    x.run(check=False)
    assert pg.paged_gqa_check_device_errors() == -5
