"""Rotary positions on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from oracle import rope as ro

pytestmark = pytest.mark.gpu


def _inv(R, base=10000.0):
    return (base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float()


def _check(got, x, pos, inv, sections, il, adj):
    """bf16 once (2^-8 of the value); the fp32 cosine and sine (2 ulp), phase (2^-25 turns, 2 pi of it) and two
    products and their sum: below 2^-20 of the pair's size."""
    ref = ro.rope(x.double().cpu().numpy(), pos.cpu().numpy(), inv.cpu().numpy(), sections, il, adj)
    size = np.abs(x.double().cpu().numpy()).max()
    off = np.abs(got.double().cpu().numpy() - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size)
    assert (off <= 0).all(), f"{(off > 0).sum()} values off, worst {off.max():.3g}"
    n = 2 * len(inv)
    assert bool((got[..., n:] == x[..., n:]).all())


CASES = [
    # T, q heads, k heads, rotated, sections, interleaved, adjacent, farthest position
    (1, 16, 1, 64, [16, 8, 8], True, False, 1000),
    (1, 1, 1, 16, [8], False, True, 10),
    (7, 24, 2, 256, [44, 42, 42], True, False, 100000),
    (33, 5, 5, 96, [12, 12, 12, 12], True, True, 2 ** 31 - 1),
    (300, 8, 1, 128, [64], False, False, 2 ** 31 - 1),
    (1000, 3, 1, 256, [0, 64, 64], False, True, 40000),
    (5000, 6, 2, 192, [32, 64], False, False, 2000000),
    (64, 0, 3, 32, [10, 6], True, False, 500),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_matches_the_oracle(i, in_place):
    T, hq, hk, R, sections, il, adj, far = CASES[i]
    g = torch.Generator().manual_seed(i)
    qkv = torch.randn(T, hq + 2 * hk, 256, generator=g).bfloat16().cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    pos = torch.randint(-far, far, (len(sections), T), generator=g, dtype=torch.int64).int().cuda()
    pos[:, 0] = 0
    inv = _inv(R).cuda()
    q0, k0, rest = q.clone(), k.clone(), qkv[:, hq + hk:].clone()
    if in_place:
        pg.paged_gqa_rope(q, k, pos, inv, sections, interleaved=il, adjacent=adj)
        qo, ko = q, k
    else:
        qo, ko = (torch.full(t.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for t in (q0, k0))
        pg.paged_gqa_rope(q, k, pos, inv, sections, qo, ko, interleaved=il, adjacent=adj)
        assert bool((q == q0).all()) and bool((k == k0).all())
    torch.cuda.synchronize()
    if hq:
        _check(qo, q0, pos, inv, sections, il, adj)
    _check(ko, k0, pos, inv, sections, il, adj)
    assert bool((qkv[:, hq + hk:] == rest).all())  # v stays


def test_extreme_positions_frequencies_and_values():
    """Frequencies from denormals to large ones at the ends of the position range."""
    inv = torch.tensor([1e-40, 1e-30, 3e-9, 1e-3, 0.5, 1.0, 6.2831855, 1234.567, 3e7, 2e-45, 0.0, 1e10, 1e-7, 0.1, 2.0, 31.4],
                       dtype=torch.float32).cuda()
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 2 ** 20]], dtype=torch.int32).cuda()
    # the oracle's extended product holds 55 bits and reduces exactly below 2^63 turns; beyond, not on every host
    ok = inv.double().cpu().numpy() < 1e5
    x = torch.randn(8, 2, 256).bfloat16().cuda()
    out, kout = torch.empty_like(x), torch.empty_like(x)
    pg.paged_gqa_rope(x, x, pos, inv, [16], out, kout, adjacent=True)
    assert bool((out == kout).all()) and bool(out.isfinite().all())
    ref = ro.rope(x.double().cpu().numpy(), pos.cpu().numpy(), inv.cpu().numpy(), [16], False, True)
    off = np.abs(out.double().cpu().numpy() - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * 8)
    for i in range(16):
        if ok[i]:
            assert (off[..., 2 * i:2 * i + 2] <= 0).all(), f"frequency {inv[i].item()}"


def test_replay_with_new_positions():
    T = 40
    x, k = torch.randn(T, 16, 256).bfloat16().cuda(), torch.randn(T, 1, 256).bfloat16().cuda()
    pos = torch.zeros(3, T, dtype=torch.int32, device="cuda")
    inv, qo, ko = _inv(64).cuda(), torch.empty_like(x), torch.empty_like(k)
    call = lambda: pg.paged_gqa_rope(x, k, pos, inv, [16, 8, 8], qo, ko)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in range(2):
        pos.copy_(torch.randint(0, 10000, (3, T), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        _check(qo, x, pos, inv, [16, 8, 8], False, False)
        _check(ko, k, pos, inv, [16, 8, 8], False, False)
