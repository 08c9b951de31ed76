"""The profiling hook around the kernels of 4-bit attention calls."""
import pytest
import torch

import paged_gqa_gb300 as pg
from tests import fp4_util as fu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [0, 1, 3])
@pytest.mark.parametrize("seqs,hq,classes", [
    ([(1, 700)] * 3, 8, (0,)),
    ([(4, 700), (1, 90)], 8, (0,)),
    ([(4, 700), (150, 900)], 16, (0, 1)),
    ([(300, 900)], 16, (0, 1)),
])
def test_events_bracket_the_kernel_of_a_class(seqs, hq, classes, path):
    c = fu.make(seqs, hq, 1, 16, seed=340)
    prev = pg.paged_gqa_set_path(path)
    try:
        for cls in classes:
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            pg.paged_gqa_set_kernel_events(cls, *ev)  # (records both once, to create them)
            torch.cuda.synchronize()
            before, after = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            before.record()
            pg.paged_gqa_attn_fp4(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out)
            after.record()
            torch.cuda.synchronize()
            assert before.elapsed_time(ev[0]) >= 0 and ev[0].elapsed_time(ev[1]) > 0 and ev[1].elapsed_time(after) >= 0
            fu.check(c, out, "with events")
            pg.paged_gqa_set_kernel_events(cls, None, None)
    finally:
        for cls in (0, 1):
            pg.paged_gqa_set_kernel_events(cls, None, None)
        pg.paged_gqa_set_path(prev)
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()
