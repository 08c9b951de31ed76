"""Block tables, tree masks, tree attention and keeping accepted tokens on the GPU, against plain loops in 64 bits."""
import random

import numpy as np
import pytest
import torch

import paged_gqa_gb300 as pg
from oracle import step
from tests import step_util as su

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------- block tables --

@pytest.mark.parametrize("S,P,W,q_hi,ctx_hi", [
    (1, 16, 40, 1, 300), (7, 16, 40, 5, 300), (33, 64, 9, 9, 500), (300, 32, 40, 4, 1200), (1025, 128, 5, 3, 600), (2500, 16, 20, 1, 300),
    (8192, 16, 6, 2, 60), (20, 16, 1300, 3, 20000), (40, 128, 300, 1, 30000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(S, P, W, q_hi, ctx_hi, in_place):
    x = su.requests(S, S, P, W, q_hi, ctx_hi)
    T = sum(n for n in x["q_lens"] if n > 0) + S % 5
    su.check_tables(x, W, T, in_place)
    su.check_tables(x, W + 3, T, in_place)  # a table wider than the pool


def test_tables_of_one_request_without_anything():
    x = dict(q_lens=[0], ctx_lens=[0], rows=[0], page_size=16, pages=[[5]], counts=[0], free=[9], num_free=1)
    su.check_tables(x, 1, 0)
    su.check_tables(x, 1, 3)


@pytest.mark.parametrize("counts_too", [False, True])
def test_tables_with_one_output_in_place(counts_too):
    x = su.requests(5, 20, 16, 30)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    t = {n: i32(x[n] if n != "num_free" else [x[n]]) for n in ("q_lens", "ctx_lens", "rows", "pages", "counts", "free", "num_free")}
    T = sum(n for n in x["q_lens"] if n > 0)
    table, lens, qsl, slots = i32([[0] * 30] * 20), i32([0] * 20), i32([0] * 21), i32([0] * T)
    counts, num = torch.zeros_like(t["counts"]), i32([0])
    pg.paged_gqa_build_tables(t["q_lens"], t["ctx_lens"], t["rows"], 16, t["pages"], t["counts"], t["free"], t["num_free"], table, lens, qsl, slots,
                              **({"page_counts_out": counts} if counts_too else {"num_free_out": num}))
    want = step.build_tables(**x, width=30, tokens=T)
    assert (counts if counts_too else t["counts"]).tolist() == want["counts"]
    assert (t["num_free"] if counts_too else num).tolist() == want["num_free"] and table.tolist() == want["table"]


def test_tables_without_requests():
    x = dict(q_lens=[], ctx_lens=[], rows=[], page_size=16, pages=[[5, 6]], counts=[1], free=[9], num_free=1)
    su.check_tables(x, 2, 4)
    su.check_tables(x, 2, 0)


@pytest.mark.parametrize("short", [1, 5, 1000])
@pytest.mark.parametrize("S", [9, 200, 1100])
def test_tables_when_pages_run_out(S, short):
    x = su.requests(100 + S, S, 16, 30, 6, 300, short=short)
    su.check_tables(x, 30, sum(n for n in x["q_lens"] if n > 0))


def test_tables_refuse_bad_requests_one_by_one():
    base = su.requests(3, 12, 16, 30, 6, 300, ended=0.2, pad=0.0)
    T = sum(n for n in base["q_lens"] if n > 0)

    def bad(tokens=T, **over):
        x = {n: ([list(y) for y in v] if n == "pages" else list(v) if isinstance(v, list) else v) for n, v in base.items()}
        for name, (i, value) in over.items():
            if i is None:
                x[name] = value
            else:
                x[name][i] = value
        su.check_tables(x, 30, tokens)

    bad(rows=(4, 99))
    bad(rows=(4, -2))
    bad(rows=(7, base["rows"][2]))  # the same row twice: the first one has it
    bad(rows=(2, base["rows"][7]))
    bad(q_lens=(5, -2))
    bad(ctx_lens=(5, -1))
    bad(ctx_lens=(5, 16 * 30 + 1), tokens=T + 50)
    bad(ctx_lens=(5, 2 ** 31 - 2))
    bad(counts=(base["rows"][6], 31))
    bad(counts=(base["rows"][6], -1))
    bad(counts=(base["rows"][6], 2 ** 31 - 1))
    bad(num_free=(None, -1))
    bad(num_free=(None, len(base["free"]) + 1))
    bad(tokens=max(0, T - 3))
    x = dict(q_lens=[-1, -1, 3], ctx_lens=[9, 9, 0], rows=[0, 1, 2], page_size=16, pages=[[1, 2], [3, 4], [0, 0]], counts=[2, 2, 0],
             free=[8, 9, -1, -1, -1], num_free=2)
    su.check_tables(x, 2, 3)  # the stack holds the first request's pages and not the second's
    x = dict(q_lens=[2, 2], ctx_lens=[0, 0], rows=[0, 1], page_size=16, pages=[[0], [0]], counts=[0, 0], free=[-5, 2 ** 28], num_free=2)
    su.check_tables(x, 1, 4)  # ids that no slot number fits


def test_tables_captured_and_replayed():
    x = su.requests(8, 40, 16, 30)
    W, T = 30, sum(n for n in x["q_lens"] if n > 0)
    dev = "cuda"
    t = {n: torch.tensor(x[n] if n != "num_free" else [x[n]], dtype=torch.int32, device=dev)
         for n in ("q_lens", "ctx_lens", "rows", "pages", "counts", "free", "num_free")}
    S = len(x["q_lens"])
    table, lens, qsl, slots = (torch.zeros(*s, dtype=torch.int32, device=dev) for s in ((S, W), (S,), (S + 1,), (T,)))
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    args = (t["q_lens"], t["ctx_lens"], t["rows"], 16, t["pages"], t["counts"], t["free"], t["num_free"], table, lens, qsl, slots)
    saved = {n: y.clone() for n, y in t.items()}
    with torch.cuda.stream(stream):
        pg.paged_gqa_build_tables(*args)
        stream.synchronize()
        for n in t:
            t[n].copy_(saved[n])
        with torch.cuda.graph(g, stream=stream):
            pg.paged_gqa_build_tables(*args)
    want = step.build_tables(**{n: ([list(y) for y in v] if n == "pages" else list(v) if isinstance(v, list) else v) for n, v in x.items()},
                             width=W, tokens=T)
    for k in range(2):  # the second replay finds every page held
        if k == 0:
            for n in t:
                t[n].copy_(saved[n])
        g.replay()
        torch.cuda.synchronize()
        assert table.tolist() == want["table"] and slots.tolist() == want["slots"] and t["num_free"].tolist() == want["num_free"]
        assert t["counts"].tolist() == want["counts"] and t["free"].tolist() == want["free"]
    assert pg.paged_gqa_check_device_errors() == 0


# ------------------------------------------------------------------------------------ tree masks --

@pytest.mark.parametrize("sizes,words,axes", [([1], 1, 1), ([5, 0, 13], 1, 2), ([32, 33, 64, 1], 2, 3), ([100, 7], 5, 4), ([1024, 1000], 32, 1)])
def test_masks(sizes, words, axes):
    r = random.Random(len(sizes))
    par = [p for n in sizes for p in su.parents(r, n)]
    if sizes[0] == 1024:
        par[:1024] = list(range(-1, 1023))  # a chain
    qsl = np.cumsum([0] + sizes).tolist()
    lens = [n + r.randint(0, 500) for n in sizes]
    T, behind = qsl[-1], 3
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    masks = torch.full((T + behind, words + 2), -7, dtype=torch.int32, device="cuda")[:, 1:1 + words]
    pos = torch.full((axes, T + behind), -7, dtype=torch.int32, device="cuda")
    pg.paged_gqa_tree_masks(i32(par + [0] * behind), i32(lens), i32(qsl), masks, pos)
    assert pg.paged_gqa_check_device_errors() == 0
    want_m, want_p = step.tree_masks(par, lens, qsl, words)
    assert masks[:T].tolist() == want_m and pos[:, :T].tolist() == [want_p] * axes
    assert (masks[T:] == -7).all() and (pos[:, T:] == -7).all()


def test_masks_flag_bad_trees():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(par, lens, qsl, words=1):
        masks = torch.full((len(par), words), -7, dtype=torch.int32, device="cuda")
        pos = torch.full((1, len(par)), -7, dtype=torch.int32, device="cuda")
        pg.paged_gqa_tree_masks(i32(par), i32(lens), i32(qsl), masks, pos)
        return masks[:, 0].tolist(), pos[0].tolist(), pg.paged_gqa_check_device_errors()

    assert run([-1, 0, 2, 9, -5], [9], [0, 5]) == ([1, 3, 4, 8, 16], [4, 5, 4, 4, 4], -5)  # not before its child: on the context
    assert run([-1, 0, 1], [2], [0, 3]) == ([0] * 3, [0] * 3, -5)  # more tokens than the sequence
    assert run([-1] + list(range(32)), [40], [0, 33])[2] == -5  # more than the mask has bits
    assert run([-1, 0, 0], [5, 5], [0, 2, 4])[2] == -5  # beyond T


# -------------------------------------------------------------------------------- tree attention --

SMALL = [
    ([(1, 1)], 4, 1, 16), ([(2, 2), (1, 90)], 8, 1, 16), ([(13, 700)], 16, 1, 16), ([(4, 130), (4, 4), (3, 257), (1, 128)], 16, 2, 32),
    ([(8, 1000), (5, 133), (8, 8)], 8, 1, 64), ([(21, 300), (10, 10)], 6, 1, 128), ([(64, 64), (64, 500), (33, 161)], 1, 1, 16),
    ([(60, 700), (4, 300), (64, 64)], 24, 2, 64), ([(130, 400), (17, 17)], 3, 1, 32), ([(5, 40)] * 70, 5, 5, 16), ([(300, 300)], 8, 2, 16),
]


@pytest.mark.parametrize("masks", ["tree", "random"])
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", range(len(SMALL)))
@pytest.mark.parametrize("path", [0, 3, 1])
def test_tree_attention(path, case, cache, masks):
    seqs, hq, hkv, P = SMALL[case]
    x = su.Tree(seqs, hq, hkv, P, cache, seed=case, masks=masks)
    prev = pg.paged_gqa_set_path(path)
    try:
        out = x.run()
        bits = pg.paged_gqa_last_plan()["path_bits"]
    finally:
        pg.paged_gqa_set_path(prev)
    assert bits & (24 if path == 1 else 6) and not bits & (6 if path == 1 else 24)
    su.compare(out, x.reference(), f"case {case} {cache} {masks}")


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_rows_that_see_nothing_are_zeros(cache):
    x = su.Tree([(5, 5), (3, 40), (130, 130), (2, 2)], 8, 2, 16, cache, masks="none")
    out = x.run()
    ref = x.reference()
    su.compare(out, ref, cache)
    for s in (0, 2, 3):
        assert (out[x.qsl[s]:x.qsl[s + 1]] == 0).all()


# (one tile each: tree calls cut longer contexts into other pieces; and the e4m3 prefill kernel rounds its exponents in
# another order on masked tiles, of which there are more in a tree call. Path 3: so few tiles would go to the prefill
# kernel, whose P is rounded otherwise than the verify kernel's)
@pytest.mark.parametrize("cache,chunk", [("e4m3", 8), ("bf16", 20)])
def test_full_masks_are_the_causal_attention_bit_for_bit(cache, chunk):
    x = su.Tree([(4, 100), (chunk, 128), (1, 33)], 16, 2, 16, cache, masks="all")
    want = torch.empty_like(x.q)
    prev = pg.paged_gqa_set_path(3)
    try:
        pg.paged_gqa_attn(x.q, x.k, x.v, x.table, x.lens_t, x.qsl_t, x.k_descale, x.v_descale, x.scale, want)
        assert torch.equal(x.run(), want)
    finally:
        pg.paged_gqa_set_path(prev)


def test_long_contexts_split_over_many_blocks():
    for cache in ("e4m3", "bf16"):
        x = su.Tree([(7, 9000), (40, 5000)], 8, 1, 64, cache, seed=4)
        su.compare(x.run(), x.reference(), cache)


def test_strided_inputs_and_wide_masks():
    x = su.Tree([(9, 300), (40, 77)], 8, 2, 16, seed=6)
    wide = torch.full((x.T, 7), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + x.words] = x.masks_t
    qq = torch.full((x.T, 10, 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    qq[:, 1:9, :256] = x.q
    big = torch.full((x.T, 9, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    out = x.run(out=big[:, :8], q=qq[:, 1:9, :256], masks=wide[:, 2:2 + x.words])
    su.compare(out, x.reference(), "strided")
    assert (big[:, 8] == 7).all()
    out = x.run(masks=wide[:, 2:6])  # words that no token has
    su.compare(out, x.reference(), "wide masks")


def test_tree_attention_captured_twice_on_two_streams():
    x = su.Tree([(13, 900), (60, 3000)], 16, 2, 16, seed=9)
    need = pg.paged_gqa_workspace_size(2, x.T, 16, 2, 16, x.table.shape[1])
    runs = []
    for _ in range(2):
        ws, out, q = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(x.q), x.q.clone()
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            pg.paged_gqa_attn_tree_ex(*x.args(q=q), out, ws)
            st.synchronize()
            with torch.cuda.graph(g, stream=st):
                pg.paged_gqa_attn_tree_ex(*x.args(q=q), out, ws)
        runs.append((g, st, out, ws, q))  # (a graph's workspace has to live as long as the graph)
    ref = x.reference()
    for k in range(3):
        for g, st, out, *_ in runs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st, out, *_ in runs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for g, st, out, *_ in runs:
            su.compare(out, ref, f"replay {k}")
    assert pg.paged_gqa_check_device_errors() == 0


def test_tree_attention_refused_in_a_capture_without_a_workspace():
    x = su.Tree([(3, 40)], 8, 1, 16)
    out = torch.empty_like(x.q)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
        with pytest.raises(pg.PagedGQAError, match="paged_gqa_attn_tree_ex"):
            pg.paged_gqa_attn_tree(*x.args(), out)


def test_calls_on_two_streams_share_the_workspace_in_turn():
    xs = [su.Tree([(13, 4000 + 100 * i), (5, 900)], 16, 1, 16, seed=i) for i in range(2)]
    outs = [torch.empty_like(x.q) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, o, st in zip(xs, outs, streams):
            with torch.cuda.stream(st):
                pg.paged_gqa_attn_tree(*x.args(), o)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        su.compare(o, x.reference(), "two streams")
    assert pg.paged_gqa_check_device_errors() == 0


def test_tree_attention_flags_what_the_masks_do_not_hold():
    x = su.Tree([(40, 100), (3, 50)], 8, 1, 16)
    out = x.run(check=False, masks=x.masks_t[:, :1].contiguous())
    assert pg.paged_gqa_check_device_errors() == -5
    assert (out[:40] == 0).all()
    ref = x.reference()
    su.compare(out[40:], ref[40:], "the other sequence")


# --------------------------------------------------------------------------------- keeping tokens --

def _keep(x, kept, num, D):
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = [(k + [99] * D)[:D] for k in kept]
    out = torch.full((len(kept),), -9, dtype=torch.int32, device="cuda")
    pg.paged_gqa_cache_keep(x.k, x.v, x.table, x.lens_t, x.qsl_t, i32(rows).reshape(len(kept), D), i32(num), out)
    return out.tolist()


def _kept_reference(x, caches, kept):
    for s, (n, L) in enumerate(x.seqs):
        ids = x.table[s].tolist()
        for c in caches:
            old = c.clone()
            for i, a in enumerate(kept[s]):
                src, dst = L - n + a, L - n + i
                c[ids[dst // x.P], dst % x.P] = old[ids[src // x.P], src % x.P]


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("seqs,hkv,P,D", [([(1, 1)], 1, 16, 1), ([(13, 300), (4, 4), (0, 20), (7, 130)], 2, 16, 5), ([(64, 64), (100, 900)], 1, 64, 40),
                                          ([(9, 40)] * 50, 3, 32, 9), ([(70, 200)], 2, 128, 70)])
def test_keep(seqs, hkv, P, D, cache):
    r = random.Random(D)
    x = su.Tree(seqs, 4 * hkv, hkv, P, cache, seed=D)
    before = [c.view(torch.uint8).clone() for c in (x.k, x.v)]
    kept = [sorted(r.sample(range(n), r.randint(0, min(n, D)))) for n, _ in seqs]
    lens = _keep(x, kept, [len(k) for k in kept], D)
    assert pg.paged_gqa_check_device_errors() == 0
    assert lens == [L - n + len(k) for (n, L), k in zip(seqs, kept)]
    _kept_reference(x, before, kept)
    for got, want in zip((x.k, x.v), before):
        assert torch.equal(got.view(torch.uint8), want)


def test_keep_flags_bad_paths_and_pages():
    x = su.Tree([(5, 30), (5, 40), (5, 50), (5, 60), (5, 70)], 4, 1, 16, seed=2)
    before = [c.view(torch.uint8).clone() for c in (x.k, x.v)]
    kept = [[0, 2], [2, 2], [1, 5], [-1, 2], [1, 4]]
    lens = _keep(x, kept, [2, 2, 2, 2, 3], 2)  # good, not increasing, outside, negative, more than D
    assert pg.paged_gqa_check_device_errors() == -5
    assert lens == [27, 35, 45, 55, 65]
    _kept_reference(x, before, [[0, 2], [], [], [], []])
    for got, want in zip((x.k, x.v), before):
        assert torch.equal(got.view(torch.uint8), want)
    x.table[0, 1] = 10 ** 6  # position 26, where the second kept token goes
    lens = _keep(x, [[1, 2], [], [], [], []], [2, 0, 0, 0, 0], 2)
    assert pg.paged_gqa_check_device_errors() == -5 and lens[0] == 27
    for got, want in zip((x.k, x.v), before):
        assert torch.equal(got.view(torch.uint8), want)


# ------------------------------------------------------------------------------ a step of them all --

def test_a_step_as_it_is_used():
    """Tables from lengths, positions and masks from parents, rotary, write, tree attention, keep; then the next step's tables."""
    r = random.Random(5)
    P, W, hq, hkv, S = 16, 20, 8, 2, 6
    ctx = [r.randint(0, 200) for _ in range(S)]
    qn = [r.randint(1, 12) for _ in range(S)]
    need = [-(-c // P) for c in ctx]
    NB = 120
    ids = r.sample(range(NB), NB)
    pages = [[-1] * W for _ in range(S + 2)]
    rows = r.sample(range(S + 2), S)
    counts = [0] * (S + 2)
    for s in range(S):
        counts[rows[s]] = need[s]
        pages[rows[s]][:need[s]], ids = ids[:need[s]], ids[need[s]:]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pages_t, counts_t, free_t, num_t = i32(pages), i32(counts), i32(ids + [-1] * (NB - len(ids))), i32([len(ids)])
    T = sum(qn)
    table, lens, qsl, slots = (torch.empty(*s, dtype=torch.int32, device="cuda") for s in ((S, W), (S,), (S + 1,), (T,)))
    pg.paged_gqa_build_tables(i32(qn), i32(ctx), i32(rows), P, pages_t, counts_t, free_t, num_t, table, lens, qsl, slots)
    par = [p for n in qn for p in su.parents(r, n)]
    masks, pos = torch.empty(T, 1, dtype=torch.int32, device="cuda"), torch.empty(1, T, dtype=torch.int32, device="cuda")
    pg.paged_gqa_tree_masks(i32(par), lens, qsl, masks, pos)
    gen = torch.Generator().manual_seed(1)
    k, v = ((torch.randn(NB, P, hkv, 256, generator=gen)).to(torch.float8_e4m3fn).cuda() for _ in range(2))
    q, kn, vn = (torch.randn(T, h, 256, generator=gen).bfloat16().cuda() for h in (hq, hkv, hkv))
    inv = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    pg.paged_gqa_rope(q, kn, pos, inv, [32])
    pg.paged_gqa_cache_write(kn, vn, k, v, table, lens, qsl, 1.0, 1.0)
    out = torch.empty_like(q)
    pg.paged_gqa_attn_tree(q, k, v, table, lens, qsl, masks, 1.0, 1.0, 1 / 16, out)
    x = su.Tree.__new__(su.Tree)
    x.seqs = [(n, c + n) for n, c in zip(qn, ctx)]
    x.T, x.hq, x.hkv, x.P, x.q, x.k, x.v, x.table, x.scale, x.k_descale, x.v_descale = T, hq, hkv, P, q, k, v, table, 1 / 16, 1.0, 1.0
    x.qsl, x.masks = qsl.tolist(), masks.tolist()
    assert x.masks == step.tree_masks(par, [L for _, L in x.seqs], x.qsl, 1)[0]
    su.compare(out, x.reference(), "step")
    # slots agree with where the write put the rows
    flat = k.view(torch.uint8).view(NB * P, hkv, 256)
    assert torch.equal(flat[slots.long()], kn.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    # accept the path to the last token of each tree
    kept = []
    for s in range(S):
        t, path = qn[s] - 1, []
        while t >= 0:
            path.append(t)
            t = par[x.qsl[s] + t]
        kept.append(path[::-1])
    D = max(map(len, kept))
    new_lens = torch.empty_like(lens)
    pg.paged_gqa_cache_keep(k, v, table, lens, qsl, i32([p + [0] * (D - len(p)) for p in kept]), i32([len(p) for p in kept]), new_lens)
    assert new_lens.tolist() == [c + len(p) for c, p in zip(ctx, kept)]
    for s in range(S):
        at = [(ctx[s] + i) for i in range(len(kept[s]))]
        where = [table[s, a // P].item() * P + a % P for a in at]
        tok = [x.qsl[s] + t for t in kept[s]]
        assert torch.equal(flat[where], kn[tok].float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    # the next step: one token each, with the pages they have
    pg.paged_gqa_build_tables(i32([1] * S), new_lens, i32(rows), P, pages_t, counts_t, free_t, num_t, table, lens, qsl, slots)
    assert lens.tolist() == [n + 1 for n in new_lens.tolist()] and qsl.tolist() == list(range(S + 1))
    assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()


# ------------------------------------------------------------------- what the calls above leave out --

def test_tables_of_more_tokens_than_31_bits_count():
    big = 2 ** 31 - 1
    x = dict(q_lens=[4, big, big, 3], ctx_lens=[5, 0, 0, 14], rows=[3, 1, 2, 0], page_size=16,
             pages=[[7], [-1], [-1], [5]], counts=[1, 0, 0, 1], free=[1, 2, 3], num_free=3)
    for row in x["pages"]:
        row += [-1]
    got, status = su.run_tables(x, 2, 9)
    assert status == -5
    assert got["lens"] == [9, 0, 0, 17] and got["qsl"] == [0, 4, big, big, big]
    assert got["slots"] == [5 * 16 + 5 + i for i in range(4)] + [-1] * 5
    assert got["table"] == [[5, -1], [-1, -1], [-1, -1], [7, 3]] and got["num_free"] == [2]


@pytest.mark.parametrize("qsl", [[2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1], [5, 2], [0, 2 ** 31 - 1], [-1, 0]])
def test_starts_from_nowhere_are_flagged(qsl):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    masks, pos = torch.full((6, 1), -7, dtype=torch.int32, device="cuda"), torch.full((1, 6), -7, dtype=torch.int32, device="cuda")
    pg.paged_gqa_tree_masks(i32([-1] * 6), i32([2 ** 31 - 1]), i32(qsl), masks, pos)
    assert pg.paged_gqa_check_device_errors() == -5
    x = su.Tree([(5, 30)], 4, 1, 16, seed=2)
    before = x.k.view(torch.uint8).clone()
    x.qsl_t = i32(qsl)
    assert _keep(x, [[1, 3]], [2], 2) == [30]
    assert pg.paged_gqa_check_device_errors() == -5 and torch.equal(before, x.k.view(torch.uint8))
    for path in (0, 3, 1):
        prev = pg.paged_gqa_set_path(path)
        try:
            x.run(check=False)
        finally:
            pg.paged_gqa_set_path(prev)
        assert pg.paged_gqa_check_device_errors() == -5


# e4m3 and bf16 caches, rows of both classes; "many": more row blocks than the verify kernel plans by itself
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("seqs,hq,hkv", [([(0, 0), (5, 60), (0, 33), (3, 3), (0, 0)], 8, 1), ([(3, 70), (1, 1), (8, 20)] * 100, 8, 2),
                                         ([(0, 9), (70, 600), (0, 1)], 4, 1)])
def test_padded_and_many_sequences(seqs, hq, hkv, cache):
    x = su.Tree(seqs, hq, hkv, 16, cache, seed=13)
    ref = x.reference()
    for path in (0, 3):
        prev = pg.paged_gqa_set_path(path)
        try:
            su.compare(x.run(), ref, f"{cache} path {path}")
        finally:
            pg.paged_gqa_set_path(prev)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("seqs,hq,hkv", [([(8, 40000)], 8, 1), ([(60, 12000)], 8, 1), ([(2, 30000), (33, 9000)], 16, 2)])
def test_blocks_of_many_pieces_and_the_same_bits_again(seqs, hq, hkv, cache):
    x = su.Tree(seqs, hq, hkv, 64, cache, seed=17)
    first = x.run()
    su.compare(first, x.reference(), cache)
    for _ in range(40):
        assert torch.equal(x.run(check=False), first)
    assert pg.paged_gqa_check_device_errors() == 0


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("seqs", [[(40, 900)], [(5, 700), (3, 90)], [(40, 900), (5, 700)], [(3, 9000)] * 3 + [(20, 5000), (1, 8000)],
                                  [(17, 40)] * 460])
def test_a_tree_wait_that_runs_out_reports_timeout_and_the_next_call_is_correct(seqs, cache):
    x = su.Tree(seqs, 8, 1, 16, cache, seed=21)
    prev = pg.paged_gqa_set_stall_test(200_000)
    try:
        x.run(check=False)
        status = pg.paged_gqa_check_device_errors()
    finally:
        pg.paged_gqa_set_stall_test(prev)
    assert status == -4, pg.paged_gqa_last_error()
    su.compare(x.run(), x.reference(), cache)


def whole_numbers(x, gen):
    """q and k as small whole numbers: scores are exact, and under a scale of 2^26 a row is V of its largest one's key."""
    for name, t in (("q", x.q), ("k", x.k)):
        setattr(x, name, torch.randint(-3, 4, t.shape, generator=gen).to(torch.bfloat16).to(t.dtype).to(t.device))
    x.scale = 2.0 ** 26


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_scores_of_2_to_the_34(path, cache):
    x = su.Tree([(40, 600), (5, 400), (3, 300)], 8, 2, 16, cache, seed=23, masks="all")
    nan = torch.isnan(x.k.float())
    whole_numbers(x, torch.Generator().manual_seed(23))
    k = x.k.float()
    x.k = k.masked_fill(nan, float("nan")).to(x.k.dtype)
    prev = pg.paged_gqa_set_path(path)
    try:
        out = x.run().float()
    finally:
        pg.paged_gqa_set_path(prev)
    seen = 0
    for s, (n, L) in enumerate(x.seqs):
        ids = x.table[s, :-(-L // 16)].long()
        for h in range(8):
            ks, vs = (c.float()[ids, :, h // 4].reshape(-1, 256)[:L] for c in (x.k, x.v))
            score = x.q[x.qsl[s]:x.qsl[s + 1], h].double() @ ks.double().T
            score = score.masked_fill(torch.arange(L, device="cuda") > L - n + torch.arange(n, device="cuda")[:, None], -1e9)
            top = score.topk(2, dim=1)
            alone = top.values[:, 0] > top.values[:, 1]
            seen += int(alone.sum())
            got, want = out[x.qsl[s]:x.qsl[s + 1], h][alone], (vs[top.indices[:, 0]] * x.v_descale)[alone]
            # V itself, except that the pieces of a split sequence are held in f16: exact from 2^-14 on (bf16 has 8
            # bits, f16 11), below that off by 2^-25, and then rounded to bf16 by at most 2^-8 of 2^-14
            small = want.abs() < 2.0 ** -14
            assert torch.equal(got[~small], want[~small])
            assert ((got - want)[small].abs() <= 2.0 ** -25 + 2.0 ** -22).all()
    assert seen > 8 * 40


def test_offsets_beyond_32_bits():
    """Caches of 10 GB each, a table, masks and rows of more than 2^31 elements apart."""
    P, hkv, NB = 128, 16, 20000
    dev = "cuda"
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device=dev)  # noqa: E731
    gen = torch.Generator().manual_seed(3)
    n, L, hq = 9, 200, 16
    ids = [19999, 19990]
    space = torch.empty(2, NB, P, hkv, 256, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    k, v = space[0], space[1]
    rows = [torch.randn(2 * P, hkv, 256, generator=gen).to(torch.float8_e4m3fn).to(dev) for _ in range(2)]
    for c, x in zip((k, v), rows):
        c[ids] = x.view(2, P, hkv, 256)
    far = torch.empty(2 * 2 ** 31 + 4096, dtype=torch.int32, device=dev)
    table = far[:2 ** 31 + 4].as_strided((2, 2), (2 ** 31, 1))
    table.copy_(i32([[0, 1], ids]))
    masks = far[8:].as_strided((n, 1), (2 ** 28 + 2 ** 10, 1))
    par = su.parents(random.Random(1), n)
    lens, qsl = i32([0, L]), i32([0, 0, n])
    pos = torch.empty(1, n, dtype=torch.int32, device=dev)
    pg.paged_gqa_tree_masks(i32(par), lens, qsl, masks, pos)
    want_masks, want_pos = step.tree_masks(par, [L], [0, n], 1)
    assert masks.tolist() == want_masks and pos.tolist() == [want_pos]
    q = torch.randn(n, hq, 256, generator=gen).bfloat16().to(dev)
    out = torch.empty_like(q)
    pg.paged_gqa_attn_tree(q, k, v, table, lens, qsl, masks, 1.0, 1.0, 1 / 16, out)
    assert pg.paged_gqa_check_device_errors() == 0
    seen = step.tree_seen(want_masks, n, L)
    ref = np.zeros((n, hq, 256))
    qd, kd, vd = q.double().cpu().numpy(), rows[0].double().cpu().numpy(), rows[1].double().cpu().numpy()
    for h in range(hq):
        ref[:, h] = step.attention(qd[:, h], kd[:L, h], vd[:L, h], seen, 1 / 16)[0]
    su.compare(out, ref, "far")
    kept = far[16:].as_strided((2, 3), (2 ** 31 + 64, 1))
    kept.copy_(i32([[0, 0, 0], [1, 4, 8]]))
    new = torch.empty(2, dtype=torch.int32, device=dev)
    pg.paged_gqa_cache_keep(k, v, table, lens, qsl, kept, i32([0, 3]), new)
    assert pg.paged_gqa_check_device_errors() == 0 and new.tolist() == [0, L - n + 3]
    for c, x in zip((k, v), rows):
        want = x.view(torch.uint8).clone()
        for i, a in enumerate([1, 4, 8]):
            want[L - n + i] = x.view(torch.uint8)[L - n + a]
        assert torch.equal(c.view(torch.uint8)[ids].view(2 * P, hkv, 256), want)
    # tables and a pool with rows that far apart
    pages, table = far.as_strided((2, 3), (2 ** 31 + 8, 1)), far[2 ** 31 + 64:].as_strided((2, 3), (2 ** 31 + 8, 1))
    pages.copy_(i32([[-1] * 3, [4, -1, -1]]))
    counts, lens, qsl, slots = i32([0, 1]), i32([0, 0]), i32([0, 0, 0]), i32([0] * 5)
    pg.paged_gqa_build_tables(i32([3, 2]), i32([0, 15]), i32([0, 1]), 16, pages, counts, i32([7, 8, 9]), i32([3]), table, lens, qsl, slots)
    assert pg.paged_gqa_check_device_errors() == 0
    assert table.tolist() == [[9, -1, -1], [4, 8, -1]] and pages.tolist() == [[9, -1, -1], [4, 8, -1]]
    assert slots.tolist() == [144, 145, 146, 79, 128]


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_keep_in_interleaved_caches(cache):
    r = random.Random(3)
    x = su.Tree([(13, 300), (40, 41)], 8, 2, 16, cache, seed=31)
    both = torch.stack([x.k.view(torch.uint8), x.v.view(torch.uint8)], dim=2).view(x.k.dtype)  # [NB, P, 2, Hkv, 256]
    before = [c.view(torch.uint8).clone() for c in (x.k, x.v)]
    x.k, x.v = both[:, :, 0], both[:, :, 1]
    su.compare(x.run(), x.reference(), "interleaved")
    kept = [sorted(r.sample(range(13), 6)), sorted(r.sample(range(40), 33))]
    assert _keep(x, kept, [6, 33], 33) == [293, 34]
    assert pg.paged_gqa_check_device_errors() == 0
    _kept_reference(x, before, kept)
    for got, want in zip((x.k, x.v), before):
        assert torch.equal(got.contiguous().view(torch.uint8), want)


def test_a_step_captured_and_replayed_against_the_eager_one():
    """Masks, tree attention, keep and the next tables in one graph, replayed on new lengths and pages."""
    x = su.Tree([(13, 300), (9, 40), (1, 1)], 8, 1, 16, seed=41)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(pg.paged_gqa_workspace_size(3, x.T, 8, 1, 16, x.table.shape[1]), dtype=torch.uint8, device="cuda")
    masks, pos = torch.empty(x.T, 1, dtype=torch.int32, device="cuda"), torch.empty(3, x.T, dtype=torch.int32, device="cuda")
    out, new, kept, num = torch.empty_like(x.q), i32([0] * 3), i32([[0, 1, 2], [0, 2, 5], [0, 0, 0]]), i32([3, 2, 1])
    k, v = (c.view(torch.uint8).clone() for c in (x.k, x.v))

    def run():
        pg.paged_gqa_tree_masks(x.parents_t, x.lens_t, x.qsl_t, masks, pos)
        pg.paged_gqa_attn_tree_ex(*x.args(masks=masks), out, ws)
        pg.paged_gqa_cache_keep(x.k, x.v, x.table, x.lens_t, x.qsl_t, kept, num, new)

    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
        st.synchronize()
        with torch.cuda.graph(g, stream=st):
            run()
    for lens, num_kept in (([300, 40, 1], [3, 2, 1]), ([290, 39, 1], [0, 3, 0]), ([13, 9, 1], [1, 1, 1])):
        x.seqs = [(n, L) for (n, _), L in zip(x.seqs, lens)]
        x.lens_t.copy_(i32(lens))
        num.copy_(i32(num_kept))
        x.k.view(torch.uint8).copy_(k)
        x.v.view(torch.uint8).copy_(v)
        ref = x.reference()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        su.compare(out, ref, lens)
        assert new.tolist() == [L - n + a for (n, L), a in zip(x.seqs, num_kept)]
        assert pg.paged_gqa_check_device_errors() == 0


def test_two_host_threads_at_once():
    import threading
    tree = su.Tree([(13, 4000), (70, 900)], 16, 2, 16, seed=51)
    prompt = su.Prompt([1500, 33], 8, 1, seed=52)
    tree_ref, failed = tree.reference(), []
    torch.cuda.synchronize()

    def work(which):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    if which:
                        out = torch.full_like(tree.q, float("nan"))
                        pg.paged_gqa_attn_tree(*tree.args(), out)
                    else:
                        out = torch.full(prompt.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
                        pg.paged_gqa_attn_prompt(prompt.q, prompt.k, prompt.v, prompt.qsl_t, prompt.scale, out)
                torch.cuda.current_stream().synchronize()
            if which:
                su.compare(out, tree_ref, "thread")
            else:
                prompt.check(out, None, rows={0: [0, 700, 1499], 1: [32]})
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert pg.paged_gqa_check_device_errors() == 0


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_calls_of_at_most_64_rows_flag_and_zero_bad_sequences_themselves(cache):
    x = su.Tree([(3, 50), (9, 400), (4, 100)], 4, 1, 16, cache, seed=61)
    ref = x.reference()
    out = x.run()
    assert pg.paged_gqa_last_plan()["path_bits"] == 2
    su.compare(out, ref, cache)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    for lens, gone in (([50, 8, 100], 1), ([2, 400, 100], 0), ([50, 400, 10 ** 6], 2), ([-1, 400, 100], 0)):
        x.lens_t = i32(lens)
        out = x.run(check=False)
        assert pg.paged_gqa_check_device_errors() == -5
        for s in range(3):
            rows = slice(x.qsl[s], x.qsl[s + 1])
            if s == gone:
                assert (out[rows] == 0).all()
            else:
                su.compare(out[rows], ref[rows], (cache, lens))
    x = su.Tree([(40, 100)], 1, 1, 16, cache, seed=62)
    out = x.run(check=False, masks=x.masks_t[:, :1].contiguous())  # 40 tokens, masks of 32
    assert pg.paged_gqa_check_device_errors() == -5 and (out == 0).all()
    x.qsl_t = i32([0, 39])  # not all of T
    x.run(check=False)
    assert pg.paged_gqa_check_device_errors() == -5


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_wide_trees_around_the_most_blocks_that_a_kernel_plans_by_itself(cache):
    for S in (1, 40, 64, 150, 230):  # 2 kv heads, 17 tokens of 4 heads: 68 rows, one block of each
        x = su.Tree([(17, 17 + 3 * s) for s in range(S)], 8, 2, 16, cache, seed=S)
        out = x.run()
        su.compare(out, x.reference(), (cache, S))
        prev = pg.paged_gqa_set_path(3)  # planned by the plan kernel
        try:
            su.compare(x.run(), x.reference(), (cache, S, "plan"))
        finally:
            pg.paged_gqa_set_path(prev)
    x = su.Tree([(300, 900), (1, 40), (0, 5), (90, 90), (700, 700)], 16, 2, 32, cache, seed=3)  # several blocks each
    su.compare(x.run(), x.reference(), cache)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_wide_trees_flag_and_zero_bad_sequences(cache):
    x = su.Tree([(30, 50), (9, 400), (40, 100)], 8, 1, 16, cache, seed=71)
    ref = x.reference()
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    for lens, gone in (([50, 8, 100], 1), ([29, 400, 100], 0), ([50, 400, 10 ** 6], 2), ([-1, 400, 100], 0)):
        x.lens_t = i32(lens)
        out = x.run(check=False)
        assert pg.paged_gqa_check_device_errors() == -5
        for s in range(3):
            rows = slice(x.qsl[s], x.qsl[s + 1])
            if s == gone:
                assert (out[rows] == 0).all()
            else:
                su.compare(out[rows], ref[rows], (cache, lens))
    # sequences that share their tokens: more blocks than tokens can have
    S, T = 121, 79
    x.lens_t, x.qsl_t = i32([100] * S), i32([0, T] * ((S + 1) // 2))
    x.table = x.table[2:3].expand(S, -1).contiguous()
    x.run(check=False)
    assert pg.paged_gqa_check_device_errors() == -5


def test_small_trees_and_wide_ones_in_one_call():
    """e4m3 caches and more than a few pages: the verify kernel with its own plan, then plan and prefill kernel."""
    x = su.Tree([(3, 9000)] * 3 + [(20, 5000)] + [(1, 8000), (2, 2), (0, 7), (8, 4000)], 8, 1, 16, seed=81)
    out = x.run()
    plan = pg.paged_gqa_last_plan()
    assert plan["path_bits"] == 6 and plan["kernels_launched"] == 4
    su.compare(out, x.reference(), "mixed")
    for _ in range(20):
        assert torch.equal(x.run(), out)
