"""Prompt attention on what its other tests leave out: many prompts of which one is bad."""
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import step_util as su

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [0, 1, "expanded"])
@pytest.mark.parametrize("lens,bad", [([3] * 70, 69), ([3] * 70, 40), ([0] * 64 + [5, 4], 65), ([200] + [2] * 300, 290)])
def test_one_bad_prompt_among_many_is_flagged(path, lens, bad):
    """Its end lies behind T, and so do all later ones'; `expanded` strides go to the warp-level kernel by themselves."""
    x = su.Prompt(lens, 8, 1, seed=70, fused=False)
    if path == "expanded":
        x.k, x.v = x.k[:1].expand(x.T, 1, 256), x.v[:1].expand(x.T, 1, 256)
    good, _ = x.run(lse=False)
    first = x.qsl[bad]
    x.qsl_t[bad + 1:] = x.T + 9
    prev = pg.paged_gqa_set_path(path if path == 1 else 0)
    try:
        out, _ = x.run(lse=False, check=False)
    finally:
        pg.paged_gqa_set_path(prev)
    assert pg.paged_gqa_check_device_errors() == -5
    assert torch.isnan(out[first:]).all()
    x.check(out, None, rows={s: list(range(n)) for s, n in enumerate(lens[:bad]) if n})
    assert good.isfinite().all()
