"""Tree attention under each of its plans: which kernels serve a call, calls whose plan does not fit, the largest number of blocks."""
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


WHICH = [  # (sequences, path, path bits, kernels): e4m3 caches, 8/2 heads
    ([(16, 600)], 0, 2, 2),                                            # the verify kernel alone, and the merge
    ([(5, 400), (3, 300), (8, 600)], 0, 2, 2),
    ([(40, 600), (5, 400), (3, 300)], 3, 6, 4),                        # plan, verify, prefill, merge
    ([(3, 9000)] * 3 + [(20, 5000)] + [(1, 8000), (2, 2), (0, 7), (8, 4000)], 0, 6, 4),  # the verify kernel plans its own class
    ([(40, 600), (5, 400), (3, 300)], 0, 4, 2),                        # the prefill kernel plans every sequence
]


@pytest.mark.parametrize("case", range(len(WHICH)))
def test_scores_of_2_to_the_34_in_every_kernel_of_e4m3_caches(case):
    seqs, path, bits, kernels = WHICH[case]
    x = su.Tree(seqs, 8, 2, 16, seed=23, masks="all")
    nan = torch.isnan(x.k.float())
    gen = torch.Generator().manual_seed(23)
    x.q = torch.randint(-3, 4, x.q.shape, generator=gen).bfloat16().cuda()  # small whole numbers: scores are exact
    x.k = torch.randint(-3, 4, x.k.shape, generator=gen).float().cuda().masked_fill(nan, float("nan")).to(x.k.dtype)
    x.scale = 2.0 ** 26
    out = _on_path(path, x.run).float()
    plan = pg.paged_gqa_last_plan()
    assert plan["path_bits"] == bits and plan["kernels_launched"] == kernels
    seen = 0
    for s, (n, L) in enumerate(x.seqs):
        ids = x.table[s, :-(-L // 16)].long()
        for h in range(8 if n else 0):
            ks, vs = (c.float()[ids, :, h // 4].reshape(-1, 256)[:L] for c in (x.k, x.v))
            score = x.q[x.qsl[s]:x.qsl[s + 1], h].double() @ ks.double().T
            score = score.masked_fill(torch.arange(L, device="cuda") > L - n + torch.arange(n, device="cuda")[:, None], -1e9)
            top = score.topk(2, dim=1)
            alone = top.values[:, 0] > top.values[:, 1]
            seen += int(alone.sum())
            got, want = out[x.qsl[s]:x.qsl[s + 1], h][alone], (vs[top.indices[:, 0]] * x.v_descale)[alone]
            # the largest score's V itself: an e4m3 value times a power of two is exact in f16 pieces and in bf16
            assert torch.equal(got, want)
    assert seen > 4 * sum(n for n, _ in seqs)


@pytest.mark.parametrize("path,bits", [(0, 4), (3, 6)])
def test_rows_that_see_nothing_are_zeros_under_each_plan(path, bits):
    x = su.Tree([(5, 5), (3, 40), (130, 130), (2, 2)], 8, 2, 16, masks="none")
    out = _on_path(path, x.run)
    assert pg.paged_gqa_last_plan()["path_bits"] == bits
    su.compare(out, x.reference(), path)
    for s in (0, 2, 3):
        assert (out[x.qsl[s]:x.qsl[s + 1]] == 0).all()
    x = su.Tree([(5, 5), (2, 40), (1, 1)], 8, 1, 16, masks="none")  # at most 64 rows: the verify kernel alone
    out = x.run()
    assert pg.paged_gqa_last_plan()["path_bits"] == 2
    su.compare(out, x.reference(), "verify")
    assert (out[:5] == 0).all() and (out[7:] == 0).all()


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


@pytest.mark.parametrize("tokens,path,bits", [(9, 0, 4), (9, 3, 4), (8, 0, 2), (8, 3, 6)])
def test_row_sums_keep_what_is_small(tokens, path, bits):
    """One key of weight 1 and 99 of 2^-12, in one tile: sum = 1 + 99 * 2^-12. V is 1 at the first key and 0 at the others,
    scaled so that the output, 1.0031, lies 0.8e-3 below the middle of two bf16 values; sums that lose seven of the
    99 (as additions in 11 bits to the first key's would) are 1.7e-3 too small, and give the other one."""
    x = su.Tree([(tokens, 100 + tokens)], 8, 1, 16, seed=5, masks="none")
    ids = x.table[0, :-(-x.lens[0] // 16)].long()
    pos = torch.arange(ids.numel() * 16, device="cuda").view(-1, 16)
    k, v = (torch.zeros(ids.numel(), 16, 1, 256, device="cuda") for _ in range(2))
    k[..., 0, 0] = torch.where(pos == 0, 0.0, -1.0)
    v[..., 0, :] = (pos == 0).float().unsqueeze(-1)
    x.k[ids], x.v[ids] = k.to(x.k.dtype), v.to(x.v.dtype)
    x.q = torch.zeros_like(x.q)
    x.q[..., 0] = 1.0
    x.k_descale, x.scale = 1.0, 12 * 0.6931471805599453
    want = (1 + 2.0 ** -8) * (1 - 0.8e-3)
    x.v_descale = want * (1 + 99 * 2.0 ** -12)
    out = _on_path(path, x.run).double()
    assert pg.paged_gqa_last_plan()["path_bits"] == bits
    # its own rounding (half a step: 2^-8), fp32's in the scales, the weights and the sums
    assert ((out - want).abs() <= 2.0 ** -8 + 2.0 ** -18).all(), (out.min(), out.max(), want)
