"""Tree attention under each of its plans: calls whose plan does not fit, the largest number of blocks."""
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


def test_more_rows_of_blocks_than_31_bits_count():
    """2^25 blocks of 64 rows: a million sequences of one token and 32 kv heads, all on the same pages."""
    S, H, L, P = 2 ** 20, 32, 380, 128
    dev = "cuda"
    gen = torch.Generator().manual_seed(4)
    k, v = (torch.randn(3, P, H, 256, generator=gen).to(torch.float8_e4m3fn).to(dev) for _ in range(2))
    q = torch.randn(1, H, 256, generator=gen).bfloat16().to(dev).expand(S, H, 256)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=dev).expand(S, 3)
    lens = torch.full((S,), L, dtype=torch.int32, device=dev)
    qsl = torch.arange(S + 1, dtype=torch.int32, device=dev)
    masks = torch.ones(1, 1, dtype=torch.int32, device=dev).expand(S, 1)
    out = torch.full((S, H, 256), float("nan"), dtype=torch.bfloat16, device=dev)
    pg.paged_gqa_attn_tree(q, k, v, table, lens, qsl, masks, 1.0, 1.0, 1 / 16, out)
    assert pg.paged_gqa_check_device_errors() == 0
    ks, vs = (c.double()[[2, 0, 1]].reshape(-1, H, 256)[:L] for c in (k, v))
    w = torch.softmax(torch.einsum("hd,khd->hk", q[0].double(), ks) / 16, 1)
    want = torch.einsum("hk,khd->hd", w, vs)
    su.compare(out[0], want.cpu().numpy(), "first")
    for i in range(0, S, 2 ** 16):  # the others differ in the order of a split block's sums at most: a bf16 step
        part = out[i:i + 2 ** 16].float()
        assert ((part - out[0].float()).abs() <= 2.0 ** -7 * out[0].float().abs() + 2.0 ** -9).all(), i
