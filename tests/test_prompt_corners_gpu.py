"""Prompt attention on what its other tests leave out: many prompts of which one is bad, statistics of NaN rows, tails next to NaN, the launch summary."""
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


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("lens,hq", [([300, 40], 8), ([9000, 3], 2)])
@pytest.mark.parametrize("which", ["q", "k"])
def test_statistics_of_rows_with_a_nan_are_nan(path, lens, hq, which):
    x = su.Prompt(lens, hq, 1, seed=71, fused=False)
    if which == "q":
        x.q[[17, 250], 1] = float("nan")
        rows = torch.zeros(x.T, hq, dtype=torch.bool, device="cuda")
        rows[[17, 250], 1] = True
    else:  # every token of the prompt from 200 on sees it
        x.k[200, 0, 5] = float("nan")
        rows = torch.zeros(x.T, hq, dtype=torch.bool, device="cuda")
        rows[200:lens[0]] = True
    prev = pg.paged_gqa_set_path(path)
    try:
        out, lse = x.run()
    finally:
        pg.paged_gqa_set_path(prev)
    assert torch.isnan(out[rows]).all() and out[~rows].isfinite().all()
    assert torch.isnan(lse[rows]).all() and lse[~rows].isfinite().all()


def test_the_launch_summary_counts_a_captured_calls_kernels():
    x = su.Prompt([300], 8, 1, seed=72)
    out = torch.empty_like(x.q)
    ws = torch.empty(pg.paged_gqa_prompt_workspace_size(1, 300, 8, 1), dtype=torch.uint8, device="cuda")
    call = lambda: pg.paged_gqa_attn_prompt_ex(x.q, x.k, x.v, x.qsl_t, x.scale, out, None, ws)  # noqa: E731
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
        st.synchronize()
        assert pg.paged_gqa_last_plan()["kernels_launched"] == 1
        with torch.cuda.graph(g, stream=st):
            call()
        assert pg.paged_gqa_last_plan()["kernels_launched"] == 2  # the epoch word moves first
        g.replay()
        st.synchronize()
    x.check(out, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (24, 2), (2, 1)])
def test_tails_next_to_nan_prompts(hq, hkv, dtype):
    """Every other prompt is NaN, so a tile that runs past its prompt's end holds V that has to be zeroed in both of a pair's
    SMs, tile after tile and in items of one tile; again and again, the same bits."""
    lens = [n for m in (1, 5, 127, 129, 31, 300, 33, 1000, 64, 2, 517, 90) for n in (m, 1 + m % 7)] * 3
    x = su.Prompt(lens, hq, hkv, dtype, seed=73)
    for s in range(1, len(lens), 2):
        for t in (x.q, x.k, x.v):
            t[x.qsl[s]:x.qsl[s + 1]] = float("nan")
    out, lse = x.run()
    x.check(out, lse, rows={s: sorted({0, n // 2, n - 1}) for s, n in enumerate(lens) if s % 2 == 0})
    good = torch.cat([torch.arange(x.qsl[s], x.qsl[s + 1]) for s in range(0, len(lens), 2)]).cuda()
    for _ in range(40):
        again, ls = x.run(check=False)
        assert torch.equal(again[good], out[good]) and torch.equal(ls[good], lse[good])
    assert pg.paged_gqa_check_device_errors() == 0
