"""Tree attention under each of its plans: calls whose plan does not fit."""
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import step_util as su

pytestmark = pytest.mark.gpu


def _on_path(path, call):
    prev = pg.paged_gqa_set_path(path)
    try:
        return call()
    finally:
        pg.paged_gqa_set_path(prev)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("path", [0, 3])
def test_a_plan_that_does_not_fit_leaves_out_as_it_was(path, cache):
    """Sequences that share their tokens make more blocks than the tokens can have: flagged, and nothing is joined from what an
    earlier call left in the workspace."""
    S, T, L = 121, 79, 1000
    x = su.Tree([(T, L)], 8, 1, 16, cache, seed=3)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    _on_path(path, x.run)  # its pieces stay behind in the workspace
    x.lens_t, x.qsl_t = i32([L] * S), i32([0, T] * ((S + 1) // 2))
    x.table = x.table.expand(S, -1).contiguous()
    out = torch.full_like(x.q, 5.0)
    _on_path(path, lambda: x.run(out=out, check=False))
    assert pg.paged_gqa_check_device_errors() == -5
    assert (out == 5).all()
