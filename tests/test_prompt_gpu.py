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
        bits = pg.paged_gqa_last_plan()["path_bits"]
    finally:
        pg.paged_gqa_set_path(prev)
    assert bits == (512 if path == 1 else 256)
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


def test_tokens_that_share_their_memory():
    """k and v of one token for all (stride 0, no tensor map for that): the warp-level kernel."""
    x = su.Prompt([40], 4, 1, seed=9, fused=False)
    x.k, x.v = x.k[:1].expand(40, 1, 256), x.v[:1].expand(40, 1, 256)
    out, lse = x.run()
    assert pg.paged_gqa_last_plan()["path_bits"] == 512
    x.check(out, lse)


def test_heads_before_tokens():
    x = su.Prompt([150, 70], 6, 3, seed=10, fused=False)
    x.q, x.k, x.v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x.q, x.k, x.v))
    out, lse = x.run()
    assert pg.paged_gqa_last_plan()["path_bits"] == 256
    x.check(out, lse)


def test_values_beyond_f16_in_split_prompts():
    x = su.Prompt([3000], 8, 1, seed=12, fused=False)
    x.v = (x.v.float() * 1e30).bfloat16()
    out, lse = x.run()
    x.check(out, lse, rows={0: [0, 500, 1500, 2999]})


def test_the_same_bits_again():
    x = su.Prompt([1900, 700, 33], 8, 2, seed=11)
    first, lse = x.run()
    for _ in range(60):
        out, ls = x.run(check=False)
        assert torch.equal(out, first) and torch.equal(ls, lse)
    assert pg.paged_gqa_check_device_errors() == 0


def test_two_captured_graphs_with_a_workspace_each():
    xs = [su.Prompt([1500 + 200 * i, 40], 8, 1, seed=20 + i) for i in range(2)]
    runs = []
    for x in xs:
        ws = torch.empty(pg.paged_gqa_prompt_workspace_size(2, x.T, 8, 1), dtype=torch.uint8, device="cuda")
        out = torch.empty(x.T, 8, 256, dtype=torch.bfloat16, device="cuda")
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            pg.paged_gqa_attn_prompt_ex(x.q, x.k, x.v, x.qsl_t, x.scale, out, None, ws)
            st.synchronize()
            with torch.cuda.graph(g, stream=st):
                pg.paged_gqa_attn_prompt_ex(x.q, x.k, x.v, x.qsl_t, x.scale, out, None, ws)
        runs.append((x, g, st, out, ws))
    for _ in range(5):
        for _, _, _, out, _ in runs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _, g, st, _, _ in runs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
    for x, _, _, out, _ in runs:
        x.check(out, None, rows={0: [0, 300, 1499], 1: [0, 39]})
    assert pg.paged_gqa_check_device_errors() == 0


def test_refused_in_a_capture_without_a_workspace():
    x = su.Prompt([40], 8, 1)
    out = torch.empty(40, 8, 256, dtype=torch.bfloat16, device="cuda")
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
        with pytest.raises(pg.PagedGQAError, match="paged_gqa_attn_prompt_ex"):
            pg.paged_gqa_attn_prompt(x.q, x.k, x.v, x.qsl_t, x.scale, out)
    with pytest.raises(pg.PagedGQAError, match="too small"):
        pg.paged_gqa_attn_prompt_ex(x.q, x.k, x.v, x.qsl_t, x.scale, out, None, torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_two_streams_and_other_calls_share_the_workspace_in_turn():
    xs = [su.Prompt([2000 - 300 * i, 9], 8, 1, seed=30 + i) for i in range(2)]
    tree = su.Tree([(13, 4000), (5, 900)], 16, 1, 16, seed=3)
    outs = [torch.empty(x.T, 8, 256, dtype=torch.bfloat16, device="cuda") for x in xs]
    tree_out = torch.empty_like(tree.q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for x, o, st in zip(xs, outs, streams):
            with torch.cuda.stream(st):
                pg.paged_gqa_attn_prompt(x.q, x.k, x.v, x.qsl_t, x.scale, o)
        with torch.cuda.stream(streams[2]):
            pg.paged_gqa_attn_tree(*tree.args(), tree_out)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        x.check(o, None, rows={0: [0, 1000, 1699], 1: [8]})
    su.compare(tree_out, tree.reference(), "tree")
    assert pg.paged_gqa_check_device_errors() == 0


def test_a_wait_that_runs_out_reports_timeout_and_the_next_call_is_correct():
    x = su.Prompt([700, 50], 8, 1, seed=40)
    prev = pg.paged_gqa_set_stall_test(200_000)
    try:
        x.run(check=False)
        status = pg.paged_gqa_check_device_errors()
    finally:
        pg.paged_gqa_set_stall_test(prev)
    assert status == -4, pg.paged_gqa_last_error()
    out, lse = x.run()
    x.check(out, lse)


def test_prompts_cut_into_many_pieces():
    x = su.Prompt([9000, 3], 2, 1, seed=50)
    out, lse = x.run()
    x.check(out, lse, rows={0: [0, 127, 128, 255, 4097, 8191, 8448, 8999], 1: [0, 2]})
    for _ in range(20):
        again, ls = x.run(check=False)
        assert torch.equal(again, out) and torch.equal(ls, lse)
    assert pg.paged_gqa_check_device_errors() == 0


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_of_2_to_the_25(path, dtype, sign):
    """q and k are small whole numbers: scores are exact, and under a scale of 2^16 a row is V of its largest one's key."""
    x = su.Prompt([600, 90], 8, 1, dtype, seed=60, fused=False)
    gen = torch.Generator().manual_seed(60)
    x.q, x.k = (torch.randint(-3, 4, t.shape, generator=gen).to(dtype).cuda() for t in (x.q, x.k))
    x.scale = sign * 2.0 ** 16
    prev = pg.paged_gqa_set_path(path)
    try:
        out, lse = x.run()
    finally:
        pg.paged_gqa_set_path(prev)
    seen = 0
    for s, n in enumerate(x.lens):
        at = x.qsl[s]
        for h in range(8):
            score = sign * (x.q[at:at + n, h].double() @ x.k[at:at + n, 0].double().T)
            score = score.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -1e9)
            top = score.topk(min(n, 2), dim=1)
            alone = top.values[:, 0] > top.values[:, 1]
            seen += int(alone.sum())
            # the row's one P is 2^x with |x| up to half a step of the reference, rounded once (u) over its unrounded self,
            # times V, rounded once (u): in f16 two halves of V's values below 2^-14 as well
            got, want = out[at:at + n, h][alone].double(), x.v[at:at + n, 0][top.indices[:, 0]][alone].double()
            assert ((got - want).abs() <= 2.1 * su.U[dtype] * want.abs() + (2.0 ** -24 if dtype is torch.float16 else 0)).all()
            # fp32 products and a rounding each: 2^-22 of the largest
            want = top.values[:, 0] * 2.0 ** 16
            assert ((lse[at:at + n, h].double() - want).abs() <= 2.0 ** -22 * want.abs() + 2.0).all()
    assert seen > 8 * 500


def test_rows_far_apart():
    """Tokens 2^28 elements apart: offsets of more than 32 bits, beyond 2^31 elements."""
    dtype, T = torch.bfloat16, 12
    x = su.Prompt([9, 3], 4, 2, dtype, seed=61, fused=False)
    step = 2 ** 28
    space = torch.empty((T - 1) * step + 4096, dtype=dtype, device="cuda")
    far = [space[i * 1024:].as_strided((T, h, 256), (step, 256, 1)) for i, h in enumerate((4, 2, 2, 4))]
    for f, t in zip(far, (x.q, x.k, x.v)):
        f.copy_(t)
    x.q, x.k, x.v = far[:3]
    out, lse = x.run(out=far[3])
    assert pg.paged_gqa_last_plan()["path_bits"] == 256
    x.check(out, lse)
    prev = pg.paged_gqa_set_path(1)
    try:
        out, lse = x.run(out=far[3].zero_())
    finally:
        pg.paged_gqa_set_path(prev)
    x.check(out, lse)


@pytest.mark.parametrize("qsl", [[0, 2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1], [0, 41, 40], [-1, 0, 0]])
@pytest.mark.parametrize("path", [0, 1])
def test_starts_from_nowhere_are_flagged(path, qsl):
    x = su.Prompt([20, 20], 8, 1, seed=62)
    x.qsl_t = torch.tensor(qsl, dtype=torch.int32, device="cuda")
    prev = pg.paged_gqa_set_path(path)
    try:
        out, _ = x.run(check=False)
    finally:
        pg.paged_gqa_set_path(prev)
    assert pg.paged_gqa_check_device_errors() == -5
    assert torch.isnan(out).all()


def test_no_prompt_at_all():
    x = su.Prompt([0, 0, 0], 8, 1, behind=30)
    out, lse = x.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()
