"""The 4-bit paged cache on the GPU: write, read, attention, and a decoding step of all of them."""
import dataclasses

import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from oracle import fp4, rope as ro
from tests import fp4_util as fu

pytestmark = pytest.mark.gpu

BOUNDS, TIMEOUT, WORKSPACE = -5, -4, -6


def _ok():
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()


def _attn(c, out=None, **kw):
    if out is None:
        out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pg.paged_gqa_attn_fp4(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out, **kw)
    return out


def _new(T, hkv, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(T, hkv, 256, generator=g) * size).bfloat16().cuda() for _ in range(2)]


# ------------------------------------------------------------------------------------ write --

WRITES = [
    # name, [(q_len, L)], kv heads, page, size of the values
    ("one token", [(1, 1)], 1, 16, 1.0),
    ("decode", [(1, 37), (1, 1), (1, 300), (1, 64), (1, 65)], 2, 16, 1.0),
    ("verify", [(4, 100), (2, 17), (3, 3), (4, 4000), (4, 18)], 1, 16, 1.0),
    ("chunks", [(300, 1200), (17, 17), (129, 500), (33, 64)], 5, 64, 1.0),
    ("whole blocks", [(32, 32), (16, 48), (160, 160)], 2, 32, 1.0),
    ("saturating", [(6, 200), (1, 9)], 2, 32, 5e4),
    ("tiny", [(21, 80)], 1, 128, 1e-5),
    ("empty sequences", [(0, 5), (3, 20), (0, 0), (2, 2), (0, 9)], 1, 16, 1.0),
]


@pytest.mark.parametrize("i", range(len(WRITES)), ids=[w[0] for w in WRITES])
def test_write_matches_the_oracle_byte_for_byte(i):
    name, seqs, hkv, page, size = WRITES[i]
    c = fu.make(seqs, hkv, hkv, page, seed=i, kd=0.0131, vd=0.0077)
    kn, vn = _new(c.T, hkv, 10 + i, size)
    ref = fp4.write(kn.float().cpu().numpy(), vn.float().cpu().numpy(), c.k.cpu().numpy(), c.v.cpu().numpy(),
                    c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
    pg.paged_gqa_cache_write_fp4(kn, vn, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd)
    _ok()
    for got, want, n in ((c.k, ref[0], "K"), (c.v, ref[1], "V")):
        bad = got.cpu().numpy() != want
        assert not bad.any(), f"{name}: {bad.sum()} {n} bytes differ, first at {np.argwhere(bad)[0]}"


def test_write_of_every_bf16_value_and_special_ones():
    """Every finite positive bf16 as one value of a group of 16 (its neighbours), their negatives in V, and
    groups with zeros, infinities and NaNs; descales that are no power of two."""
    bits = torch.arange(0, 0x8000, dtype=torch.int32)  # NaNs and infinity among them
    vals = (bits << 16).view(torch.float32).bfloat16()
    n = vals.numel() // 256
    kn = vals.view(n, 1, 256).cuda()
    vn = (-vals.float()).bfloat16().view(n, 1, 256).flip(0).contiguous().cuda()
    vn[0, 0, :] = 0
    vn[1, 0, 5] = float("nan")
    vn[2, 0, 37] = float("-inf")
    vn[3, 0, :] = float("-inf")
    c = fu.make([(n, n + 5)], 1, 1, 16, seed=40)
    for kd, vd in ((1.7, 0.3), (1.0, 2.0 ** -100), (1e30, 1e-20)):
        ref = fp4.write(kn.float().cpu().numpy(), vn.float().cpu().numpy(), c.k.cpu().numpy(), c.v.cpu().numpy(),
                        c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), kd, vd)
        pg.paged_gqa_cache_write_fp4(kn, vn, c.k, c.v, c.table, c.lens, c.qsl, kd, vd)
        _ok()
        for got, want, is_v in ((c.k, ref[0], False), (c.v, ref[1], True)):
            g, w = fp4.unpack(got.cpu().numpy(), is_v), fp4.unpack(want, is_v)
            assert (g[1] == w[1]).all(), "scales"
            real = ~np.isnan(fp4.values(*w))  # the codes under a NaN scale say nothing
            assert (g[0][real] == w[0][real]).all(), "codes"


def test_write_and_read_of_strided_views_in_one_allocation():
    """K and V of one allocation [NB, 2, Hkv, P, 144] and of one projection's output [T, 2 Hkv, 256]."""
    seqs, hkv, page = [(19, 50), (3, 40), (16, 16)], 2, 32
    c = fu.make(seqs, hkv, hkv, page, seed=50)
    both = torch.full((c.k.shape[0], 2, hkv, page, 144), 7, dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    kv = torch.randn(c.T, 2 * hkv + 1, 256).bfloat16().cuda()
    kn, vn = kv[:, :hkv], kv[:, hkv:2 * hkv]
    ref = fp4.write(kn.float().cpu().numpy(), vn.float().cpu().numpy(), c.k.cpu().numpy(), c.v.cpu().numpy(),
                    c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
    pg.paged_gqa_cache_write_fp4(kn, vn, both[:, 0], both[:, 1], c.table, c.lens, c.qsl, c.kd, c.vd)
    assert (both[:, 0].cpu().numpy() == ref[0]).all() and (both[:, 1].cpu().numpy() == ref[1]).all()
    out = torch.full((c.T, 2 * hkv + 1, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    pg.paged_gqa_cache_read_fp4(both[:, 0], both[:, 1], c.table, c.lens, c.qsl, c.kd, c.vd, out[:, :hkv], out[:, hkv:2 * hkv])
    _ok()
    want = fp4.read(*ref, c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
    for got, w in ((out[:, :hkv], want[0]), (out[:, hkv:2 * hkv], want[1])):
        assert (np.abs(got.double().cpu().numpy() - w) <= 2.0 ** -8 * np.abs(w)).all()
    assert bool((out[:, 2 * hkv] == 3.0).all())  # the rows between stay as they were


# ------------------------------------------------------------------------------------- read --

@pytest.mark.parametrize("i,kd", [(0, 0.25), (1, 0.0131), (2, 0.0131), (3, 4.0), (4, 0.1), (7, 0.5)])
def test_read_matches_the_oracle(i, kd):
    name, seqs, hkv, page, _ = WRITES[i]
    c = fu.make(seqs, hkv, hkv, page, seed=60 + i, kd=kd, vd=2 * kd)
    k = torch.full((c.T, hkv, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    pg.paged_gqa_cache_read_fp4(c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, k, v)
    _ok()
    want = fp4.read(c.k.cpu().numpy(), c.v.cpu().numpy(), c.table.cpu().numpy(), c.lens.cpu().numpy(),
                    c.qsl.cpu().numpy(), c.kd, c.vd)
    exact = np.log2(kd) == int(np.log2(kd))
    for got, w in ((k, want[0]), (v, want[1])):
        g = got.double().cpu().numpy()
        # one rounding to fp32 (2^-24) and one to bf16; none at all under a power of two
        assert (np.abs(g - w) <= (0 if exact else (2.0 ** -8 + 2.0 ** -23)) * np.abs(w)).all(), name


def test_bad_places_are_flagged_skipped_and_read_as_zeros():
    c = fu.make([(2, 30), (20, 40), (1, 20)], 1, 1, 16, seed=70)
    kn, vn = _new(c.T, 1, 70)
    table, lens = c.table.clone(), c.lens.clone()
    table[0, 1] = c.k.shape[0] + 5   # the page of sequence 0's new tokens
    lens[1] = 10                     # 20 new tokens of 10 in all
    k0, v0 = c.k.cpu().numpy(), c.v.cpu().numpy()
    pg.paged_gqa_cache_write_fp4(kn, vn, c.k, c.v, table, lens, c.qsl, c.kd, c.vd)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    ref = fp4.write(kn[22:].float().cpu().numpy(), vn[22:].float().cpu().numpy(), k0, v0, c.table[2:].cpu().numpy(),
                    c.lens[2:].cpu().numpy(), np.array([0, 1]), c.kd, c.vd)
    assert (c.k.cpu().numpy() == ref[0]).all() and (c.v.cpu().numpy() == ref[1]).all()
    k = torch.full((c.T, 1, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    pg.paged_gqa_cache_read_fp4(c.k, c.v, table, lens, c.qsl, c.kd, c.vd, k, v)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    assert bool((k[:22] == 0).all()) and bool((v[:22] == 0).all()) and bool((k[22] != 0).any())


# -------------------------------------------------------------------------------- attention --

ATTN = [
    # name, [(q_len, L)], q heads, kv heads, page
    ("one key", [(1, 1)], 16, 1, 16),
    ("one token", [(1, 600)], 16, 1, 16),
    ("decode", [(1, 37), (1, 128), (1, 129), (1, 1000), (1, 5)], 8, 1, 64),
    ("decode two heads", [(1, 300), (1, 17)], 32, 2, 16),
    ("verify", [(4, 700), (2, 90), (3, 1500), (4, 4), (1, 255)], 16, 1, 16),
    ("verify 128-token pages", [(4, 1000), (3, 129), (2, 127), (1, 128)], 24, 2, 128),
    ("one head per kv head", [(4, 200), (1, 65)], 5, 5, 32),
    ("three heads", [(4, 333), (1, 1)], 3, 1, 32),
    ("full verify block", [(4, 257), (4, 64)], 32, 2, 16),
    ("wide group", [(1, 300), (2, 70)], 48, 1, 16),
    ("a token over the verify rows", [(1, 200), (2, 33)], 72, 1, 16),
    ("prefill", [(150, 400)], 8, 1, 64),
    ("fresh prefill", [(130, 130), (65, 65)], 16, 2, 16),
    ("mixed", [(4, 300), (129, 700), (1, 50), (0, 20), (33, 33), (2, 1000)], 24, 2, 64),
    ("empty sequences", [(0, 0), (2, 40), (0, 100), (1, 9)], 16, 1, 16),
    ("long", [(4, 20000), (1, 9999)], 16, 1, 16),
    ("single tokens, long", [(1, 30000), (1, 7777), (1, 16), (1, 17), (1, 31)], 16, 1, 32),
    ("single tokens, groups of eight", [(1, 5000), (1, 1), (1, 640), (1, 129)], 16, 2, 128),
    ("single tokens, small groups", [(1, 1000), (1, 33), (1, 257)], 12, 4, 16),
    ("as many tokens as sequences, unevenly", [(0, 40), (3, 700), (0, 0), (1, 300), (4, 129), (0, 9), (0, 8), (1, 5), (0, 3)], 16, 1, 16),
    ("the same in groups of eight", [(0, 40), (3, 700), (0, 0), (1, 300), (4, 129), (0, 9), (0, 8), (1, 5), (0, 3)], 8, 1, 16),
    ("single tokens and a prefill chunk of idle sequences' tokens", [(12, 2000)] + [(0, 30 + i) for i in range(11)] + [(1, 77)], 8, 1, 16),
    ("more blocks than a self-planned launch takes", [(1, 1 + 5 * (i % 40)) for i in range(180)], 24, 3, 16),
    ("as many of verify steps", [(1 + i % 3, 4 + 7 * (i % 40)) for i in range(180)], 24, 3, 16),
]


@pytest.mark.parametrize("path", [1, 0, 2, 3])
@pytest.mark.parametrize("i", range(len(ATTN)), ids=[a[0] for a in ATTN])
def test_attention_matches_the_oracle(i, path):
    name, seqs, hq, hkv, page = ATTN[i]
    c = fu.make(seqs, hq, hkv, page, seed=80 + i)
    prev = pg.paged_gqa_set_path(path)
    try:
        out = _attn(c)
    finally:
        pg.paged_gqa_set_path(prev)
    _ok()
    fu.check(c, out, name)


PATHS = [
    # seqs, q heads, kv heads, path: bits of the kernels that run (2 tcgen05 verify, 4 tcgen05 prefill, 128 decode)
    ([(1, 300)] * 3, 8, 1, 0, 128),
    ([(1, 300)] * 3, 8, 1, 2, 2),
    ([(1, 300)] * 3, 9, 1, 0, 2),
    ([(2, 300)], 8, 1, 0, 2),
    ([(9, 300)], 8, 1, 0, 2 | 4),
    ([(1, 300)] * 9, 8, 1, 0, 128 | 4),
]


@pytest.mark.parametrize("i", range(len(PATHS)))
def test_kernel_of_a_batch(i):
    seqs, hq, hkv, path, bits = PATHS[i]
    c = fu.make(seqs, hq, hkv, 16, seed=170 + i)
    prev = pg.paged_gqa_set_path(path)
    try:
        out = _attn(c)
    finally:
        pg.paged_gqa_set_path(prev)
    _ok()
    assert pg.paged_gqa_last_plan()["path_bits"] == bits
    fu.check(c, out, "kernel of a batch")


@pytest.mark.parametrize("name,seqs,hq", [
    ("decode", [(1, 3000), (1, 129), (1, 5)], 8),
    ("verify", [(4, 3000), (2, 700), (3, 129)], 16),
    ("prefill", [(150, 400), (4, 9000), (40, 300)], 8),
])
def test_a_wait_that_runs_out_reports_timeout_and_the_next_call_is_correct(name, seqs, hq):
    c = fu.make(seqs, hq, 1, 16, seed=180)
    prev = pg.paged_gqa_set_stall_test(200_000)  # 200 us
    try:
        _attn(c)
        st = pg.paged_gqa_check_device_errors()
    finally:
        pg.paged_gqa_set_stall_test(prev)
    assert st == TIMEOUT, pg.paged_gqa_last_error()
    out = _attn(c)
    _ok()
    fu.check(c, out, f"after a timeout ({name})")


@pytest.mark.parametrize("seqs,hq,hkv,page", [
    ([(2000, 9000)], 8, 1, 64),                                       # every CTA walks many tiles of many blocks
    ([(611, 9001), (4, 8800), (574, 8900), (1, 777), (537, 5000)] + [(3, 3000)] * 9, 24, 2, 64),
    ([(1500, 1500), (1, 12000)], 5, 5, 16),
])
def test_long_chunks_on_sampled_rows(seqs, hq, hkv, page):
    c = fu.make(seqs, hq, hkv, page, seed=99)
    rows = np.unique(np.concatenate([np.random.default_rng(7).integers(0, c.T * hq, 1500), np.arange(hq), c.T * hq - 1 - np.arange(hq)]))
    for _ in range(3):
        out = _attn(c)
        _ok()
        fu.check(c, out, "long chunks", rows=rows)


def test_large_and_small_scores():
    """Scores of hundreds (one key takes the whole row) and queries of very different sizes in one block."""
    c = fu.make([(4, 500), (1, 300)], 16, 1, 16, seed=100, size=4.0, kd=0.05)
    size = torch.logspace(-20, 1, 16, base=10.0).view(1, 16, 1)
    c.q = (c.q.float().cpu() * size).bfloat16().cuda()
    fu.check(c, _attn(c), "sizes")
    _ok()
    c.q.zero_()
    fu.check(c, _attn(c), "zero queries")


def test_rows_of_later_tokens_and_other_rows_stay_apart():
    """A NaN query row makes that row NaN and no other; a NaN key makes NaN of the rows that see it and,
    for K, of no others."""
    c = fu.make([(4, 300), (2, 77)], 16, 1, 16, seed=101)
    c.q[1, 3, 7] = float("nan")
    out = _attn(c)
    _ok()
    assert bool(out[1, 3].isnan().all())
    c.q[1, 3, 7] = 0.0
    rows = [r for r in range(6 * 16) if r != 16 + 3]
    fu.check(c, out, "other rows", rows=np.array(rows))
    # position 298 of sequence 0 is seen by its tokens 2 and 3 only
    page = int(c.table[0, 298 // 16])
    c.k[page, 0, 298 % 16, 128 + 4] = 0x7F
    out = _attn(c)
    _ok()
    assert bool(out[2:4].isnan().all()) and bool(out[[0, 1, 4, 5]].isfinite().all())
    fu.check(c, out, "rows before the NaN key", rows=np.array([r for r in range(96) if not 32 <= r < 64]))


def test_rows_of_no_sequence_stay_as_they_were_and_views_work():
    c = fu.make([(3, 100), (2, 50)], 8, 2, 32, seed=102)
    wide_q = torch.zeros(c.T, 12, 256, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 2:10] = c.q
    wide_out = torch.full((c.T, 10, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    c.q = wide_q[:, 2:10]
    both = torch.zeros(c.k.shape[0], 2, *c.k.shape[1:], dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[:, 3:3 + c.table.shape[1]] = c.table
    pg.paged_gqa_attn_fp4(c.q, both[:, 0], both[:, 1], table[:, 3:3 + c.table.shape[1]], c.lens, c.qsl, c.kd, c.vd,
                          c.scale, wide_out[:, 1:9])
    _ok()
    fu.check(c, wide_out[:, 1:9], "views")
    assert bool((wide_out[:, [0, 9]] == 5.0).all())


def test_invalid_single_token_sequences_are_zeroed_and_flagged():
    c = fu.make([(1, 100), (1, 60), (1, 400)], 8, 1, 16, seed=106)
    lens, table = c.lens.clone(), c.table.clone()
    lens[1] = 0                       # fewer than its new tokens
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pg.paged_gqa_attn_fp4(c.q, c.k, c.v, c.table, lens, c.qsl, c.kd, c.vd, c.scale, out)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    assert bool((out[1] == 0).all())
    rows = np.array([r for r in range(24) if not 8 <= r < 16])
    fu.check(c, out, "valid single tokens", rows=rows)
    table[0, 2], table[2, 20] = -7, c.k.shape[0]
    pg.paged_gqa_attn_fp4(c.q, c.k, c.v, table, c.lens, c.qsl, c.kd, c.vd, c.scale, out)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    fu.check(c, out, "the sequence with good pages", rows=np.arange(8, 16))


def test_invalid_sequences_are_zeroed_and_flagged():
    c = fu.make([(4, 100), (3, 60), (2, 40)], 16, 1, 16, seed=103)
    lens = c.lens.clone()
    lens[1] = 2  # fewer than its new tokens
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pg.paged_gqa_attn_fp4(c.q, c.k, c.v, c.table, lens, c.qsl, c.kd, c.vd, c.scale, out)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    assert bool((out[4:7] == 0).all())
    rows = np.array([r for r in range(9 * 16) if not 64 <= r < 112])
    fu.check(c, out, "valid sequences", rows=rows)


def test_bad_page_is_flagged_and_other_sequences_are_right():
    c = fu.make([(4, 100), (3, 60)], 16, 1, 16, seed=104)
    table = c.table.clone()
    table[0, 2], table[0, 3] = -7, c.k.shape[0]
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pg.paged_gqa_attn_fp4(c.q, c.k, c.v, table, c.lens, c.qsl, c.kd, c.vd, c.scale, out)
    assert pg.paged_gqa_check_device_errors() == BOUNDS
    fu.check(c, out, "the other sequence", rows=np.arange(64, 112))


def test_calls_on_other_streams_and_growing_batches():
    """Calls in a row on three streams, with batches that grow the workspace, each right."""
    streams = [torch.cuda.Stream() for _ in range(2)] + [torch.cuda.default_stream()]
    cases = [fu.make([(4, 900 + 300 * i)] * (2 + 5 * i), 16, 1, 16, seed=110 + i) for i in range(4)]
    torch.cuda.synchronize()
    outs = []
    for r in range(3):
        for i, c in enumerate(cases):
            s = streams[(r + i) % 3]
            out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            if i % 2:
                _attn(c, out, stream=s)
            else:
                with torch.cuda.stream(s):
                    _attn(c, out)
            outs.append((c, out))
    torch.cuda.synchronize()
    _ok()
    for c, out in outs:
        fu.check(c, out, "streams")


def test_two_threads_at_once():
    """Calls of two host threads, each on its own stream, in the library's workspace and in one of each thread's."""
    import threading
    cases = [fu.make([(1, 9000), (4, 700)], 16, 1, 16, seed=140), fu.make([(1, 2000)] * 6, 8, 1, 64, seed=141)]
    want = [_attn(c) for c in cases]
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in cases]

    def run(c, w, stream):
        with torch.cuda.stream(stream):
            ws = _workspace(c)
            for i in range(40):
                out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
                if i % 2:
                    _attn(c, out)
                else:
                    pg.paged_gqa_attn_fp4_ex(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out, ws)
                if not bool((out == w).all()):
                    wrong.append(i)
    threads = [threading.Thread(target=run, args=a) for a in zip(cases, want, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _ok()
    assert not wrong
    for c, w in zip(cases, want):
        fu.check(c, w, "threads")


def _far(t, step):
    """t's values in a view whose first axis steps far: `step` elements."""
    buf = torch.empty(step * (t.shape[0] - 1) + t[0].numel(), dtype=t.dtype, device="cuda")
    v = buf.as_strided(t.shape, (step, *t[0].contiguous().stride()))
    v.copy_(t)
    return v


@pytest.mark.parametrize("seqs,hq", [([(4, 50), (1, 33)], 16), ([(1, 60), (1, 20)], 8), ([(70, 75)], 8)])
def test_offsets_beyond_32_bits(seqs, hq):
    """Pages a gigabyte apart, query rows more than 2^32 bytes apart from first to last: the whole step."""
    c = fu.make(seqs, hq, 1, 16, seed=150)
    gap = (5 * 2 ** 30 // (c.k.shape[0] - 1) + 15) // 16 * 16
    c.k, c.v = _far(c.k, gap), _far(c.v, gap)
    gap = (2 ** 32 // 2 // (c.T - 1) + 256) // 8 * 8 + 256 * hq
    kn, vn = (_far(x, gap) for x in _new(c.T, 1, 151))
    want = fp4.write(kn.float().cpu().numpy(), vn.float().cpu().numpy(), c.k.contiguous().cpu().numpy(), c.v.contiguous().cpu().numpy(),
                     c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
    pg.paged_gqa_cache_write_fp4(kn, vn, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd)
    _ok()
    assert (c.k.contiguous().cpu().numpy() == want[0]).all() and (c.v.contiguous().cpu().numpy() == want[1]).all()
    pg.paged_gqa_cache_read_fp4(c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, kn, vn)
    back = fp4.read(*want, c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
    for x, w in ((kn, back[0]), (vn, back[1])):
        assert (np.abs(x.double().cpu().numpy() - w) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w)).all()
    c.q = _far(c.q, gap)
    out = _far(torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda"), gap)
    pos = torch.arange(c.T, dtype=torch.int32, device="cuda")[None]
    inv = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()
    q0 = c.q.double().cpu().numpy()
    pg.paged_gqa_rope(c.q, kn, pos, inv, [32], c.q, torch.empty(c.T, 1, 256, dtype=torch.bfloat16, device="cuda"))
    ref = ro.rope(q0, pos.cpu().numpy(), inv.cpu().numpy(), [32], False, False)
    assert (np.abs(c.q.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.abs(q0).max()).all()
    for path in (0, 1):
        out.fill_(float("nan"))
        prev = pg.paged_gqa_set_path(path)
        try:
            _attn(c, out)
        finally:
            pg.paged_gqa_set_path(prev)
        _ok()
        fu.check(dataclasses.replace(c, q=c.q.contiguous(), k=c.k.contiguous(), v=c.v.contiguous()), out, "far apart")


def test_sequences_that_share_pages():
    """Three sequences on one prefix (the same pages in every table row), each with its own last page."""
    c = fu.make([(2, 700), (2, 700), (1, 690)], 16, 1, 32, seed=142)
    c.table[1:, :20] = c.table[0, :20]
    _ok()
    fu.check(c, _attn(c), "shared prefix")
    c.table[2] = c.table[1]  # and two of them in all of them
    fu.check(c, _attn(c), "shared pages")
    _ok()


def test_results_repeat_bit_for_bit():
    c = fu.make([(4, 9000), (2, 30000), (300, 900)], 16, 1, 16, seed=120)
    a, b = _attn(c), _attn(c)
    assert bool((a.view(torch.int16) == b.view(torch.int16)).all())


def _workspace(c):
    n = pg.paged_gqa_workspace_size(len(c.seqs), c.T, c.hq, c.hkv, c.page, c.table.shape[1], torch.cuda.current_device())
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def test_capture_needs_the_callers_workspace():
    c = fu.make([(4, 500)], 16, 1, 16, seed=130)
    out = _attn(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(pg.PagedGQAError) as e:
        with torch.cuda.graph(graph):
            _attn(c, out)
    assert e.value.status == WORKSPACE
    ws = _workspace(c)
    with pytest.raises(pg.PagedGQAError):
        pg.paged_gqa_attn_fp4_ex(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out, ws[:-256])
    with pytest.raises(pg.PagedGQAError):
        pg.paged_gqa_attn_fp4_ex(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out, None)


@pytest.mark.parametrize("seqs,hq", [([(1, 30000)], 8), ([(4, 30000)], 16), ([(1, 20000)] * 4, 8), ([(1, 9000), (4, 5000), (30, 700)], 16)])
def test_replays_and_direct_calls_share_a_workspace(seqs, hq):
    """Split sequences, replayed with new queries and called directly in between, in one workspace of any contents."""
    c = fu.make(seqs, hq, 1, 16, seed=131)
    ws = _workspace(c).fill_(255)
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    call = lambda: pg.paged_gqa_attn_fp4_ex(c.q, c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, out, ws)
    call()
    fu.check(c, out, "first")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for r in range(3):
        c.q.copy_(c.q * -0.75 + 0.25)
        out.fill_(float("nan"))
        graph.replay()
        fu.check(c, out, f"replay {r}")
        out.fill_(float("nan"))
        call()
        fu.check(c, out, f"call {r}")
    _ok()


def _step(c, x, ws, buf):
    """One decoding step: rotary, cache write, attention; and the new tokens read back."""
    pg.paged_gqa_rope(x["q"], x["k"], x["pos"], x["inv"], [16, 8, 8], buf["q"], buf["k"], interleaved=True)
    pg.paged_gqa_cache_write_fp4(buf["k"], x["v"], c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd)
    pg.paged_gqa_attn_fp4_ex(buf["q"], c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, c.scale, buf["out"], ws)
    pg.paged_gqa_cache_read_fp4(c.k, c.v, c.table, c.lens, c.qsl, c.kd, c.vd, buf["kb"], buf["vb"])


@pytest.mark.parametrize("captured", [False, True])
def test_decoding_steps_of_all_operators_together(captured):
    """Three steps of a batch (single tokens, verify steps, a chunk), each against the oracles' chain; captured
    once and replayed with new inputs and lengths."""
    seqs = [(1, 600), (4, 1500), (150, 400), (2, 33)]
    c = fu.make([(q, L + 300) for q, L in seqs], 16, 2, 16, seed=140, kd=0.01, vd=0.01)
    T, g = c.T, torch.Generator().manual_seed(5)
    x = dict(q=torch.zeros(T, 16, 256, dtype=torch.bfloat16, device="cuda"), pos=torch.zeros(3, T, dtype=torch.int32, device="cuda"),
             inv=(10000.0 ** -(torch.arange(0, 64, 2) / 64)).float().cuda())
    x["k"], x["v"] = (torch.zeros(T, 2, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    buf = dict(q=torch.empty_like(x["q"]), k=torch.empty_like(x["k"]), out=torch.empty_like(x["q"]),
               kb=torch.empty_like(x["k"]), vb=torch.empty_like(x["v"]))
    ws = _workspace(c)
    c.lens.copy_(torch.tensor([L for _, L in seqs], dtype=torch.int32))
    step = lambda: _step(c, x, ws, buf)  # noqa: E731
    if captured:
        k0, v0 = c.k.clone(), c.v.clone()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        c.k.copy_(k0)
        c.v.copy_(v0)
        step = graph.replay
    for n in range(3):
        lens = torch.tensor([L + n * 7 for _, L in seqs], dtype=torch.int32)
        c.lens.copy_(lens)
        for name in ("q", "k", "v"):
            x[name].copy_(torch.randn(x[name].shape, generator=g).bfloat16())
        x["pos"].copy_(torch.randint(0, 5000, (3, T), generator=g, dtype=torch.int32))
        k0, v0 = c.k.cpu().numpy(), c.v.cpu().numpy()
        step()
        torch.cuda.synchronize()
        _ok()
        turned = {m: ro.rope(x[m].double().cpu().numpy(), x["pos"].cpu().numpy(), x["inv"].cpu().numpy(), [16, 8, 8], True, False)
                  for m in ("q", "k")}
        for m in ("q", "k"):  # bf16 once; fp32 products and phases: 2^-21 of the pair
            off = np.abs(buf[m].double().cpu().numpy() - turned[m])
            assert (off <= 2.0 ** -8 * np.abs(turned[m]) + 2.0 ** -20 * 8).all()
        ref = fp4.write(buf["k"].float().cpu().numpy(), x["v"].float().cpu().numpy(), k0, v0, c.table.cpu().numpy(),
                        c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
        assert (c.k.cpu().numpy() == ref[0]).all() and (c.v.cpu().numpy() == ref[1]).all()
        c.q = buf["q"]
        fu.check(c, buf["out"], f"step {n}")
        want = fp4.read(*ref, c.table.cpu().numpy(), c.lens.cpu().numpy(), c.qsl.cpu().numpy(), c.kd, c.vd)
        for got, w in ((buf["kb"], want[0]), (buf["vb"], want[1])):
            assert (np.abs(got.double().cpu().numpy() - w) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w)).all()
