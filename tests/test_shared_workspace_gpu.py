"""Captured calls that use one workspace in turn: a replay finds in it whatever the calls before it left."""
import pytest
import torch

import paged_gqa_gb300 as pg
import workloads as wl
from tests import fp4_util as fu
from tests import step_util as su

pytestmark = pytest.mark.gpu


def _capture(call):
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
        st.synchronize()
        with torch.cuda.graph(g, stream=st):
            call()
    torch.cuda.synchronize()
    return g


def _verify():
    """(q, out, eager call, call with a workspace, workspace bytes) of 64 verify steps of 4 tokens, split over the SMs."""
    spec = wl.config_spec(2)
    c = wl.make_case(spec, device="cuda", seed=1)
    a = (c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, c.query_start_loc)
    out = torch.empty_like(c.q)
    need = pg.paged_gqa_workspace_size(64, spec.total_q, 16, 1, 16, c.block_table.shape[1])
    return (c.q, out, lambda o: pg.paged_gqa_attn(*a, c.k_descale, c.v_descale, c.softmax_scale, o),
            lambda ws: pg.paged_gqa_attn_ex(*a, 1.0, c.k_descale, c.v_descale, c.softmax_scale, out, ws), need)


def _fp4():
    c = fu.make([(4, 5000 + 700 * i) for i in range(12)] + [(1, 900)] * 3, 16, 1, 16, seed=5)
    a = (c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale)
    out = torch.empty_like(c.q)
    need = pg.paged_gqa_workspace_size(15, c.T, 16, 1, 16, c.table.shape[1])
    return c.q, out, lambda o: pg.paged_gqa_attn_fp4(*a, o), lambda ws: pg.paged_gqa_attn_fp4_ex(*a, out, ws), need


def _tree():
    x = su.Tree([(13, 9000), (60, 12000), (2, 300)], 16, 2, 16, seed=9)
    out = torch.empty_like(x.q)
    need = pg.paged_gqa_workspace_size(3, x.T, 16, 2, 16, x.table.shape[1])
    return x.q, out, lambda o: pg.paged_gqa_attn_tree(*x.args(), o), lambda ws: pg.paged_gqa_attn_tree_ex(*x.args(), out, ws), need


def _replay_and_compare(q, out, eager, graph, gen, before=None):
    for k in range(3):
        if before is not None:
            before()
        q.copy_(torch.randn(q.shape, generator=gen).to(q.dtype))
        out.fill_(float("nan"))
        want = torch.empty_like(out)
        eager(want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()


@pytest.mark.parametrize("other", [_verify, _fp4, _tree])
def test_a_prompt_and_another_call_captured_on_one_workspace(other):
    """The prompt is the same at every replay, so it leaves the same bytes behind each time."""
    gen = torch.Generator().manual_seed(7)
    prompt = su.Prompt([16384], 16, 2, seed=3)
    q, out, eager, call, need = other()
    ws = torch.empty(max(need, pg.paged_gqa_prompt_workspace_size(1, prompt.T, 16, 2)), dtype=torch.uint8, device="cuda")
    p_out = torch.empty(prompt.q.shape, dtype=torch.bfloat16, device="cuda")
    p_args = (prompt.q, prompt.k, prompt.v, prompt.qsl_t, prompt.scale)
    p_graph = _capture(lambda: pg.paged_gqa_attn_prompt_ex(*p_args, p_out, None, ws))
    graph = _capture(lambda: call(ws))
    p_want = torch.empty_like(p_out)
    pg.paged_gqa_attn_prompt(*p_args, p_want)

    def before():
        p_out.fill_(float("nan"))
        p_graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p_out, p_want)
    _replay_and_compare(q, out, eager, graph, gen, before)


def test_two_shapes_of_one_call_captured_on_one_workspace():
    """A verify batch and a wider one of the same entry point, whose workspaces are laid out for their own sizes."""
    gen = torch.Generator().manual_seed(8)
    q, out, eager, call, need = _verify()
    x = su.Tree([(200, 9000), (90, 4000)], 16, 1, 16, seed=11, masks="all")
    wide = torch.empty_like(x.q)
    a = x.args()[:6]
    need2 = pg.paged_gqa_workspace_size(2, x.T, 16, 1, 16, x.table.shape[1])
    ws = torch.empty(max(need, need2), dtype=torch.uint8, device="cuda")
    second = _capture(lambda: pg.paged_gqa_attn_ex(*a, 1.0, x.k_descale, x.v_descale, x.scale, wide, ws))
    graph = _capture(lambda: call(ws))
    _replay_and_compare(q, out, eager, graph, gen, lambda: (second.replay(), torch.cuda.synchronize()))


def _prompt():
    x = su.Prompt([9000, 700], 4, 1, seed=13, fused=False)
    out = torch.empty_like(x.q)
    need = pg.paged_gqa_prompt_workspace_size(2, x.T, 4, 1)
    a = (x.q, x.k, x.v, x.qsl_t, x.scale)
    return x.q, out, lambda o: pg.paged_gqa_attn_prompt(*a, o), lambda ws: pg.paged_gqa_attn_prompt_ex(*a, out, None, ws), need


@pytest.mark.parametrize("which", [_verify, _fp4, _tree, _prompt])
def test_a_program_that_uses_the_workspace_between_replays(which):
    """It writes the same values over the first bytes each time; the rest stays as the last replay left it."""
    gen = torch.Generator().manual_seed(9)
    q, out, eager, call, need = which()
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = _capture(lambda: call(ws))
    _replay_and_compare(q, out, eager, graph, gen, lambda: ws[:256].fill_(7))
