"""A step of speculative decoding with token trees, and attention over whole prompts: the cases they are measured on.

  tables   block tables and slot maps from request lengths, with the page pool they draw from
  masks    ancestor masks and positions of the new tokens from their tree's parents
  tree     attention of a tree of drafted tokens over the paged cache
  keep     the drafted tokens' K and V written to the cache, then the accepted ones moved into their final places
  prompt   causal attention over whole packed prompts of different lengths, without a cache

`run` with `own` false computes each from elementary torch operations (float32 and int64); with `own` true it makes
the calls of paged_gqa_gb300 (include/paged_gqa.h says what each computes).
"""
import math

import torch

own = False

D = 256


# ------------------------------------------------------------------------------------------ cases --

def listed():
    return [
        # one verify step of a decoding batch padded for a captured graph: 1 to 4 tokens a request, long contexts, small pages
        dict(name="tables_decode", op="tables", reqs=250, admit=0, ended=3, pad=6, q_hi=4, new_hi=1, ctx_hi=32768, page=16, width=2080),
        # a busy step: many requests, new prompts admitted, others ended
        dict(name="tables_admit", op="tables", reqs=1500, admit=41, ended=37, pad=0, q_hi=1, new_hi=4096, ctx_hi=8192, page=64, width=160),
        # a few small trees: latency
        dict(name="masks_small", op="masks", seqs=7, q_lo=5, q_hi=13, words=1, axes=1),
        # a wide batch of 64-node trees, positions on three axes
        dict(name="masks_wide", op="masks", seqs=256, q_lo=17, q_hi=64, words=2, axes=3),
        # one sequence with one small tree on a bf16 cache: the latency of a single user
        dict(name="tree_one", op="tree", cache="bf16", seqs=1, q_lo=13, q_hi=13, l_lo=700, l_hi=700, hq=16, hkv=1, page=16, random=False),
        # small trees for a batch with ragged contexts: the cache's bytes count
        dict(name="tree_batch", op="tree", cache="e4m3", seqs=64, q_lo=5, q_hi=8, l_lo=1024, l_hi=32768, hq=16, hkv=2, page=16, random=False),
        # wide trees: hundreds of rows share each key, the products count
        dict(name="tree_wide", op="tree", cache="e4m3", seqs=32, q_lo=33, q_hi=60, l_lo=2048, l_hi=16384, hq=16, hkv=2, page=64, random=False),
        # accepting a few tokens of a few sequences: latency
        dict(name="keep_small", op="keep", seqs=5, q_lo=4, q_hi=13, l_lo=300, l_hi=900, hkv=1, page=16, most=4),
        # the largest step: 64 drafted tokens a sequence, up to seven accepted
        dict(name="keep_batch", op="keep", seqs=256, q_lo=33, q_hi=64, l_lo=256, l_hi=1024, hkv=2, page=64, most=7),
        # the prompt of a chat's first turn: latency
        dict(name="prompt_short", op="prompt", type="bf16", seqs=1, l_lo=173, l_hi=173, hq=8, hkv=1, lse=False),
        # prompts of very different lengths packed into one call, with the statistics a later merge needs
        dict(name="prompt_packed", op="prompt", type="f16", seqs=24, l_lo=1, l_hi=2500, hq=24, hkv=2, lse=True),
        # one long document: bound by the matrix products
        dict(name="prompt_long", op="prompt", type="bf16", seqs=1, l_lo=16384, l_hi=16384, hq=16, hkv=2, lse=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "masks", "tree", "tree", "tree", "keep", "prompt", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        reqs = _log_int(rng, 1, 2000)
        ctx = _log_int(rng, 1, min(32768, 4000000 // reqs))
        new = _log_int(rng, 1, 4096)
        return dict(op=op, reqs=reqs, admit=rng.randint(0, max(1, reqs // 8)), ended=rng.randint(0, reqs // 8), pad=rng.choice([0, 0, rng.randint(1, 40)]),
                    q_hi=rng.choice([1, 4, 9]), new_hi=new, ctx_hi=ctx, page=page, width=-(-max(ctx + 9, new) // page) + rng.randint(0, 9))
    if op == "masks":
        words = rng.choice([1, 2, 3, 8])
        q_hi = rng.randint(1, 32 * words)
        return dict(op=op, seqs=_log_int(rng, 1, 512), q_lo=rng.randint(1, q_hi), q_hi=q_hi, words=words, axes=rng.choice([1, 2, 3, 4]))
    if op == "keep":
        seqs, q_hi = _log_int(rng, 1, 200), _log_int(rng, 1, 64)
        l_hi = q_hi + _log_int(rng, 1, min(4096, 200000 // seqs))
        return dict(op=op, seqs=seqs, q_lo=rng.randint(1, q_hi), q_hi=q_hi, l_lo=rng.randint(q_hi, l_hi), l_hi=l_hi, hkv=rng.choice([1, 2]), page=page,
                    most=rng.randint(1, min(16, q_hi)))
    hq, hkv = rng.choice([(8, 1), (16, 1), (32, 2), (24, 2), (6, 1), (12, 1), (8, 4), (3, 1), (5, 5)])
    if op == "tree":
        seqs, q_hi = _log_int(rng, 1, 96), _log_int(rng, 2, 100)
        cache = rng.choice(["e4m3", "e4m3", "bf16"])
        l_hi = q_hi + _log_int(rng, 1, min(30000, max(64, 3000000 // (seqs * q_hi)), max(64, 1900000 // (seqs * hkv * (2 if cache == "bf16" else 1)))))
        return dict(op=op, cache=cache, seqs=seqs, q_lo=rng.randint(1, q_hi), q_hi=q_hi, l_lo=rng.randint(q_hi, l_hi), l_hi=l_hi,
                    hq=hq, hkv=hkv, page=page, random=rng.random() < 0.4)
    seqs = _log_int(rng, 1, 48)
    l_hi = _log_int(rng, 1, int(math.sqrt(2e9 / hq / seqs)))
    return dict(op=op, type=rng.choice(["bf16", "bf16", "f16"]), seqs=seqs, l_lo=rng.randint(1, l_hi), l_hi=l_hi, hq=hq, hkv=hkv, lse=rng.random() < 0.5)


def _between(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen).tolist()


def _lengths(case):
    """[(q_len, L)] of the batch: the same for every seed, so that `work` can count them."""
    gen = torch.Generator().manual_seed(30 + case["seqs"] + 7 * case["l_hi"])
    if case["op"] == "prompt":
        return [(n, n) for n in _between(gen, case["l_lo"], case["l_hi"], case["seqs"])]
    seqs = zip(_between(gen, case["q_lo"], case["q_hi"], case["seqs"]), _between(gen, case["l_lo"], case["l_hi"], case["seqs"]))
    return [(min(q, n), n) for q, n in seqs]


def _tree_sizes(case):
    return _between(torch.Generator().manual_seed(40 + case["seqs"] + 7 * case["q_hi"]), case["q_lo"], case["q_hi"], case["seqs"])


def _requests(case):
    """(new tokens, cached tokens, pages held beyond those) of each request: new -1 where it has ended."""
    gen = torch.Generator().manual_seed(50 + case["reqs"] + 7 * case["ctx_hi"])
    n = case["reqs"]
    q, ctx = _between(gen, 1, case["q_hi"], n), _between(gen, 1, case["ctx_hi"], n)
    spare = _between(gen, 0, 1, n)
    kind = torch.randperm(n, generator=gen).tolist()
    new = _between(gen, 1, case["new_hi"], n)
    for i in range(n):
        if kind[i] < case["admit"]:
            q[i], ctx[i], spare[i] = new[i], 0, 0
        elif kind[i] >= n - case["ended"]:
            q[i] = -1
    # a spare page, left by tokens that were rejected, fits the table's row
    most = case["width"]
    spare = [min(s, most - -(-c // case["page"])) if s else 0 for s, c in zip(spare, ctx)]
    return q, ctx, spare


def work(case):
    if case["op"] == "tables":
        q, ctx, _ = _requests(case)
        P, S = case["page"], case["reqs"] + case["pad"]
        pages = sum(-(-(c + n) // P) for n, c in zip(q, ctx) if n >= 0)
        taken = sum(-(-(c + n) // P) - -(-c // P) for n, c in zip(q, ctx) if n >= 0)
        given = sum(-(-c // P) for n, c in zip(q, ctx) if n < 0)
        total = sum(max(n, 0) for n in q) + case["pad"]
        return {"bytes": 4 * (3 * S + S + 2 * S + 1 + pages + S * case["width"] + 3 * taken + 2 * given + total), "flops": 4 * total}
    if case["op"] == "masks":
        q = _tree_sizes(case)
        return {"bytes": 4 * sum(q) * (1 + case["words"] + case["axes"]) + 8 * len(q), "flops": sum(q) * case["words"]}
    seqs = _lengths(case)
    T = sum(q for q, _ in seqs)
    if case["op"] == "prompt":
        pairs = sum(n * (n + 1) // 2 for _, n in seqs)
        return {"bytes": T * D * 2 * (2 * case["hq"] + 2 * case["hkv"]) + (T * case["hq"] * 4 if case["lse"] else 0), "flops": 4 * D * case["hq"] * pairs}
    tables = sum(-(-n // case["page"]) for _, n in seqs) * 4 + len(seqs) * 8
    if case["op"] == "tree":
        size = 2 if case["cache"] == "bf16" else 1
        pairs = sum(q * (n - q + 1) for q, n in seqs)  # the context and the token itself, at least
        return {"bytes": sum(n for _, n in seqs) * case["hkv"] * 2 * D * size + T * case["hq"] * D * 4 + tables + T * 4 * _words(case), "flops": 4 * D * case["hq"] * pairs}
    moved = sum(len(k) for k in _kept(case))
    return {"bytes": T * case["hkv"] * 2 * D * 3 + moved * case["hkv"] * 2 * D * 2 + T * 4 + len(seqs) * (12 + 4 * case["most"]), "flops": T * case["hkv"] * 2 * D}


def _words(case):
    return -(-case["q_hi"] // 32)


# ----------------------------------------------------------------------------------------- inputs --

def _parents(sizes, gen):
    """A random tree for each size, in one list: token 0 hangs on the context, the others on an earlier one (often the latest)."""
    got = []
    for n in sizes:
        r = torch.rand(n, generator=gen).tolist()
        got += [-1] + [i - 1 if r[i] < 0.3 else int(r[i] * 37 * i) % i for i in range(1, n)]
    return got


def _kept(case):
    """Each sequence's accepted tokens: the same for every seed. Increasing, as the tokens of one path are."""
    gen = torch.Generator().manual_seed(60 + case["seqs"] + 7 * case["l_hi"])
    got = []
    for q, _ in _lengths(case):
        n = int(torch.randint(0, min(case["most"], q) + 1, (1,), generator=gen))
        got.append(sorted(torch.randperm(q, generator=gen)[:n].tolist()))
    return got


def _seen(parents, qsl, q_max):
    """bool [S, q_max, q_max]: does token i of a sequence have token j on its path (itself among it)?"""
    S = qsl.numel() - 1
    qn = (qsl[1:] - qsl[:-1]).long()
    t = torch.arange(q_max, device=parents.device)
    at = (qsl[:-1].long().unsqueeze(1) + t).clamp(max=parents.numel() - 1)
    par = parents.long()[at]
    real = t < qn.unsqueeze(1)
    seen = torch.zeros(S, q_max + 1, q_max, dtype=torch.bool, device=parents.device)  # the last row stands for the context
    s = torch.arange(S, device=parents.device)
    for i in range(q_max):
        p = par[:, i]
        seen[:, i] = seen[s, torch.where(p >= 0, p, torch.full_like(p, q_max))]
        seen[:, i, i] = True
    return seen[:, :q_max] & real.unsqueeze(2), real, at


def _pack_bits(seen, words):
    """bool [..., n] -> int32 [..., words], bit i of word w is value 32 w + i."""
    seen = torch.nn.functional.pad(seen, (0, 32 * words - seen.shape[-1]))
    x = (seen.unflatten(-1, (words, 32)).long() << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).int()


def _tables(case, seqs, gen, dev):
    """Pages in random order for each sequence; entries past its own are -1."""
    P = case["page"]
    need = torch.tensor([-(-n // P) for _, n in seqs], device=dev)
    NB, W = int(need.sum()) + 3, int(need.max()) + 1
    order = torch.randperm(NB, generator=gen, device=dev).int()
    table = torch.full((len(seqs), W), -1, dtype=torch.int32, device=dev)
    held = torch.arange(W, device=dev) < need.unsqueeze(1)
    table[held] = order[:NB - 3]
    return table, NB


def _cache(case, gen, NB, dev, table, lens, poison):
    """K and V caches; slots that no sequence holds are NaN where `poison` is."""
    P, H = case["page"], case["hkv"]
    kind = torch.bfloat16 if case.get("cache") == "bf16" else torch.float8_e4m3fn
    held = torch.zeros(NB, P, dtype=torch.bool, device=dev)
    slots = torch.arange(table.shape[1] * P, device=dev).view(1, -1, P) < lens.view(-1, 1, 1)
    real = table >= 0
    held[table[real].long()] = slots[real]
    caches = []
    for descale, big in ((case["kd"], 0.5), (case["vd"], 0.0)):
        buf = torch.empty(NB, P, H, D, dtype=kind, device=dev)
        # some channels of K are larger than others, as in trained models
        size = torch.exp(big * torch.randn(D, generator=gen, device=dev))
        step = max(1, (1 << 26) // (H * P * D))
        for b in range(0, NB, step):
            x = torch.randn(min(step, NB - b), P, H, D, generator=gen, device=dev) * size / descale
            if poison:
                x = torch.where(held[b:b + step, :, None, None], x.clamp(-448, 448), torch.full_like(x, math.nan))
            else:
                x = x.clamp(-448, 448)
            buf[b:b + step] = x.to(kind)
        caches.append(buf)
    return caches


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, gen, dev)
    if case["op"] == "masks":
        sizes = _tree_sizes(case)
        T = sum(sizes)
        qsl = torch.tensor([0] + sizes, device=dev).cumsum(0).int()
        lens = torch.tensor(sizes, device=dev, dtype=torch.int32) + torch.randint(0, 30000, (len(sizes),), generator=gen, device=dev, dtype=torch.int32)
        return dict(case=case, parents=torch.tensor(_parents(sizes, host), dtype=torch.int32, device=dev), qsl=qsl, lens=lens, q_max=max(sizes),
                    masks=torch.empty(T, case["words"], dtype=torch.int32, device=dev), positions=torch.empty(case["axes"], T, dtype=torch.int32, device=dev))
    seqs = _lengths(case)
    T = sum(q for q, _ in seqs)
    qsl = torch.tensor([0] + [q for q, _ in seqs], device=dev).cumsum(0).int()
    if case["op"] == "prompt":
        kind = torch.bfloat16 if case["type"] == "bf16" else torch.float16
        hq, hkv = case["hq"], case["hkv"]
        qkv = torch.randn(T, hq + 2 * hkv, D, generator=gen, device=dev)
        qkv[:, hq:hq + hkv] *= torch.exp(0.5 * torch.randn(D, generator=gen, device=dev))
        qkv = qkv.to(kind)  # one projection's output
        return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], qsl=qsl, out=torch.empty(T, hq, D, dtype=kind, device=dev),
                    lse=torch.empty(T, hq, dtype=torch.float32, device=dev) if case["lse"] else None)
    lens = torch.tensor([n for _, n in seqs], dtype=torch.int32, device=dev)
    table, NB = _tables(case, seqs, gen, dev)
    kd, vd = (2.0 ** -float(x) for x in torch.randint(3, 6, (2,), generator=host))
    if case.get("cache") == "bf16":
        kd = vd = 1.0
    case = dict(case, kd=kd, vd=vd)
    k, v = _cache(case, gen, NB, dev, table, lens, poison=case["op"] == "tree")
    s = dict(case=case, k=k, v=v, table=table, lens=lens, qsl=qsl, q_max=max(q for q, _ in seqs))
    if case["op"] == "keep":
        s["k_new"], s["v_new"] = (torch.randn(T, case["hkv"], D, generator=gen, device=dev).bfloat16() for _ in range(2))
        kept = _kept(case)
        s["kept"] = torch.tensor([x + [-1] * (case["most"] - len(x)) for x in kept], dtype=torch.int32, device=dev)
        s["num"] = torch.tensor([len(x) for x in kept], dtype=torch.int32, device=dev)
        s["lens_out"] = torch.empty_like(lens)
        return s
    if case["random"]:  # masks that are no tree's: bits of later tokens (not used) and rows that see no new token among them
        bits = torch.rand(T, 32 * _words(case), generator=gen, device=dev) < torch.rand(T, 1, generator=gen, device=dev).round() * 0.5
        s["masks"] = _pack_bits(bits, _words(case))
    else:
        parents = torch.tensor(_parents([q for q, _ in seqs], host), dtype=torch.int32, device=dev)
        seen, real, _ = _seen(parents, qsl, s["q_max"])
        s["masks"] = _pack_bits(seen[real], _words(case))
    s["q"] = torch.randn(T, case["hq"], D, generator=gen, device=dev).bfloat16()
    s["out"] = torch.empty_like(s["q"])
    return s


def _prepare_tables(case, gen, dev):
    q, ctx, spare = (torch.tensor(x, device=dev) for x in _requests(case))
    n, P, W = case["reqs"], case["page"], case["width"]
    S, R = n + case["pad"], n + 5
    held = (ctx + P - 1) // P + spare
    taken = torch.where(q >= 0, ((ctx + q + P - 1) // P - held).clamp(min=0), torch.zeros_like(q))
    NB = int(held.sum() + taken.sum()) + 11
    ids = torch.randperm(NB, generator=gen, device=dev).int()
    rows = torch.randperm(R, generator=gen, device=dev)[:n]
    pages = torch.full((R, W), -1, dtype=torch.int32, device=dev)
    counts = torch.zeros(R, dtype=torch.int32, device=dev)
    counts[rows] = held.int()
    mine = torch.arange(W, device=dev) < counts.unsqueeze(1)
    used = int(held.sum())
    pages[mine] = ids[:used]
    free = torch.full((NB,), -1, dtype=torch.int32, device=dev)
    free[:NB - used] = ids[used:]
    fill = torch.full((case["pad"],), -1, device=dev)
    total = int(q.clamp(min=0).sum()) + case["pad"]

    def int32(*x):
        return torch.cat(x).int()

    def new(*shape):
        return torch.empty(*shape, dtype=torch.int32, device=dev)

    return dict(case=case, q_lens=int32(q, fill * 0), ctx_lens=int32(ctx, fill * 0), rows=int32(rows, fill), pages=pages, counts=counts, free=free,
                num_free=torch.tensor([NB - used], dtype=torch.int32, device=dev), table=new(S, W), lens=new(S), qsl=new(S + 1), slots=new(total),
                counts_out=new(R), num_free_out=new(1))


# -------------------------------------------------------------------------------------- the passes --

def run(s):
    if own:
        return _own(s)
    return {"tables": _plain_tables, "masks": _plain_masks, "tree": _plain_tree, "keep": _plain_keep, "prompt": _plain_prompt}[s["case"]["op"]](s)


def _own(s):
    import paged_gqa_gb300 as pg
    c = s["case"]
    if c["op"] == "tables":
        pg.paged_gqa_build_tables(s["q_lens"], s["ctx_lens"], s["rows"], c["page"], s["pages"], s["counts"], s["free"], s["num_free"],
                                  s["table"], s["lens"], s["qsl"], s["slots"], s["counts_out"], s["num_free_out"])
        return _tables_of(s)
    if c["op"] == "masks":
        pg.paged_gqa_tree_masks(s["parents"], s["lens"], s["qsl"], s["masks"], s["positions"])
        return {"masks": s["masks"], "positions": s["positions"]}
    if c["op"] == "tree":
        pg.paged_gqa_attn_tree(s["q"], s["k"], s["v"], s["table"], s["lens"], s["qsl"], s["masks"], c["kd"], c["vd"], 1 / 16, s["out"])
        return {"out": s["out"]}
    if c["op"] == "keep":
        pg.paged_gqa_cache_write(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], s["qsl"], c["kd"], c["vd"])
        pg.paged_gqa_cache_keep(s["k"], s["v"], s["table"], s["lens"], s["qsl"], s["kept"], s["num"], s["lens_out"])
        return {"k": s["k"], "v": s["v"], "lens": s["lens_out"]}
    pg.paged_gqa_attn_prompt(s["q"], s["k"], s["v"], s["qsl"], 1 / 16, s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}


def _tables_of(s):
    return {"table": s["table"], "lens": s["lens"], "qsl": s["qsl"], "slots": s["slots"], "pages": s["pages"], "counts": s["counts_out"],
            "free": s["free"], "num_free": s["num_free_out"]}


def _plain_tables(s):
    P, W = s["case"]["page"], s["pages"].shape[1]
    q, ctx, row = s["q_lens"].long(), s["ctx_lens"].long(), s["rows"].long()
    pages, counts, free = s["pages"], s["counts"].long(), s["free"]
    live = row >= 0
    ended = live & (q < 0)
    act = live & (q >= 0)
    at = row.clamp(min=0)
    zero = torch.zeros_like(q)
    have = counts[at]
    j = torch.arange(W, device=q.device)
    # ended requests give their pages back
    given = torch.where(ended, have, zero)
    to = (s["num_free"].long() + given.cumsum(0) - given).unsqueeze(1) + j
    back = j < given.unsqueeze(1)
    free[to[back]] = pages[at][back]
    there = s["num_free"].long() + given.sum()
    # the others take what they need from the top of the stack
    new = torch.where(act, q, zero)
    length = torch.where(act, ctx + new, zero)
    need = (length + P - 1) // P
    take = torch.where(act, (need - have).clamp(min=0), zero)
    first = take.cumsum(0) - take
    ok = act & ((take == 0) | (first + take <= there))
    took = torch.where(ok, take, zero)
    got = ok.unsqueeze(1) & (j >= have.unsqueeze(1)) & (j < need.unsqueeze(1))
    src = there - 1 - (first.unsqueeze(1) + j - have.unsqueeze(1))
    pages[at.unsqueeze(1).expand(-1, W)[got], j.expand(at.numel(), -1)[got]] = free[src[got]]
    counts[at[ended]] = 0
    counts[at[ok]] = (have + took)[ok]
    s["counts_out"].copy_(counts)
    s["num_free_out"].copy_(there - took.sum())
    s["table"].copy_(torch.where(ok.unsqueeze(1) & (j < need.unsqueeze(1)), pages[at], torch.full_like(pages[at], -1)))
    s["lens"].copy_(torch.where(ok, length, zero))
    s["qsl"][0] = 0
    s["qsl"][1:] = new.cumsum(0)
    t = torch.arange(s["slots"].numel(), device=q.device)
    seq = torch.searchsorted(s["qsl"].long(), t, right=True) - 1
    real = seq < q.numel()
    seq = seq.clamp(max=q.numel() - 1)
    pos = ctx[seq] + t - s["qsl"][seq].long()
    slot = pages[at[seq], (pos // P).clamp(max=W - 1)].long() * P + pos % P
    s["slots"].copy_(torch.where(real & ok[seq], slot, torch.full_like(slot, -1)))
    return _tables_of(s)


def _plain_masks(s):
    seen, real, at = _seen(s["parents"], s["qsl"], s["q_max"])
    s["masks"][at[real]] = _pack_bits(seen, s["case"]["words"])[real]
    depth = seen.sum(-1) - 1
    pos = (s["lens"].long() - (s["qsl"][1:] - s["qsl"][:-1]).long()).unsqueeze(1) + depth
    s["positions"][:, at[real]] = pos[real].int()
    return {"masks": s["masks"], "positions": s["positions"]}


def _plain_tree(s):
    c = s["case"]
    H, G, P = c["hkv"], c["hq"] // c["hkv"], c["page"]
    dev = s["q"].device
    pages = s["table"].clamp(min=0).long()
    S, W = pages.shape
    n = W * P
    j = torch.arange(n, device=dev)
    held = (j < s["lens"].unsqueeze(1))[:, None, :, None]
    k = s["k"][pages].transpose(2, 3).transpose(1, 2).flatten(2, 3).float().masked_fill(~held, 0.0)  # [S, H, n, 256]
    v = s["v"][pages].transpose(2, 3).transpose(1, 2).flatten(2, 3).float().masked_fill(~held, 0.0)
    # the new tokens of each sequence, padded to the most; token t sees the context and, of the new tokens 0 .. t, those of its mask
    t = torch.arange(s["q_max"], device=dev)
    qn = (s["qsl"][1:] - s["qsl"][:-1]).long()
    real = t < qn.unsqueeze(1)
    token = (s["qsl"][:-1].long().unsqueeze(1) + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][token].float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [S, H, q_max * G, 256]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(c["kd"] / 16)
    ctx = s["lens"].long() - qn
    i = j - ctx.unsqueeze(1)  # the new token that key j is
    words = s["masks"][token].long()  # [S, q_max, words]
    w = (i // 32).clamp(0, words.shape[2] - 1).unsqueeze(1).expand(-1, s["q_max"], -1)
    bit = (words.gather(2, w) >> (i % 32).unsqueeze(1)) & 1
    seen = (i.unsqueeze(1) < 0) | ((i.unsqueeze(1) <= t.unsqueeze(1)) & (bit == 1))
    p.masked_fill_(~seen.repeat_interleave(G, 1).unsqueeze(1), -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30) * c["vd"]
    o = o.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).flatten(2, 3).bfloat16()
    out = torch.zeros_like(s["q"])
    out[token[real]] = o[real]
    return {"out": out}


def _plain_keep(s):
    c = s["case"]
    T, P = s["k_new"].shape[0], c["page"]
    t = torch.arange(T, device=s["qsl"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["qsl"], t, right=True) - 1
    pos = (s["lens"][seq] - (s["qsl"][seq + 1] - t)).long()
    page, slot = s["table"][seq, pos // P].long(), pos % P
    ctx = (s["lens"] - (s["qsl"][1:] - s["qsl"][:-1])).long()
    n = torch.arange(c["most"], device=t.device)
    move = n < s["num"].unsqueeze(1)
    which = torch.arange(ctx.numel(), device=t.device).unsqueeze(1).expand(-1, c["most"])[move]
    src, dst = (ctx.unsqueeze(1) + s["kept"])[move], (ctx.unsqueeze(1) + n)[move]
    for new, cache, descale in ((s["k_new"], s["k"], c["kd"]), (s["v_new"], s["v"], c["vd"])):
        rows = cache.view(torch.uint8)
        rows[page, slot] = (new.float() * (1.0 / descale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        rows[s["table"][which, dst // P].long(), dst % P] = rows[s["table"][which, src // P].long(), src % P]
    return {"k": s["k"], "v": s["v"], "lens": (ctx + s["num"]).int()}


def _plain_prompt(s):
    c = s["case"]
    hkv, G = c["hkv"], c["hq"] // c["hkv"]
    out, lse = s["out"], s["lse"]
    at = 0
    for n, _ in _lengths(c):
        j = torch.arange(n, device=out.device)
        hidden = j > j.unsqueeze(1)
        for h in range(hkv):
            q = s["q"][at:at + n, h * G:(h + 1) * G].float().transpose(0, 1)
            k, v = (s[x][at:at + n, h].float() for x in ("k", "v"))
            p = torch.matmul(q, k.t()).mul_(1 / 16).masked_fill_(hidden, -math.inf)
            m = p.amax(-1, keepdim=True)
            total = p.sub_(m).exp_().sum(-1, keepdim=True)
            out[at:at + n, h * G:(h + 1) * G] = (torch.matmul(p, v) / total).transpose(0, 1).to(out.dtype)
            if lse is not None:
                lse[at:at + n, h * G:(h + 1) * G] = (m + total.log()).squeeze(-1).t()
        at += n
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


# ------------------------------------------------------------------- the definition, in 64 bits --

def exact(case, seed):
    return {"tables": _exact_tables, "masks": _exact_masks, "tree": _exact_tree, "keep": _exact_keep, "prompt": _exact_prompt}[case["op"]](prepare(case, seed))


def _exact_tables(s):
    """Request by request, with lists."""
    P, W = s["case"]["page"], s["table"].shape[1]
    q, ctx, rows = s["q_lens"].tolist(), s["ctx_lens"].tolist(), s["rows"].tolist()
    pages, counts, free = s["pages"].tolist(), s["counts"].tolist(), s["free"].tolist()
    top = int(s["num_free"])
    for n, r in zip(q, rows):
        if r >= 0 and n < 0:
            for i in range(counts[r]):
                free[top] = pages[r][i]
                top += 1
            counts[r] = 0
    table, lens, qsl, slots = [], [], [0], []
    for n, c, r in zip(q, ctx, rows):
        if r < 0 or n < 0:
            table.append([-1] * W)
            lens.append(0)
            qsl.append(qsl[-1])
            continue
        need = -(-(c + n) // P)
        while counts[r] < need:
            top -= 1
            pages[r][counts[r]] = free[top]
            counts[r] += 1
        table.append(pages[r][:need] + [-1] * (W - need))
        lens.append(c + n)
        qsl.append(qsl[-1] + n)
        slots += [pages[r][i // P] * P + i % P for i in range(c, c + n)]
    slots += [-1] * (s["slots"].numel() - len(slots))
    got = {"table": table, "lens": lens, "qsl": qsl, "slots": slots, "pages": pages, "counts": counts, "free": free, "num_free": [top]}
    return {name: torch.tensor(x) for name, x in got.items()}


def _exact_masks(s):
    parents, qsl, lens = s["parents"].tolist(), s["qsl"].tolist(), s["lens"].tolist()
    masks, positions = [], []
    for i, n in enumerate(lens):
        q0, q1 = qsl[i], qsl[i + 1]
        for t in range(q1 - q0):
            path, at = 0, t
            depth = -1
            while at >= 0:
                path |= 1 << at
                at = parents[q0 + at]
                depth += 1
            row = [(path >> (32 * w)) & 0xFFFFFFFF for w in range(s["case"]["words"])]
            masks.append([x - (1 << 32) if x >= 1 << 31 else x for x in row])
            positions.append(n - (q1 - q0) + depth)
    return {"masks": torch.tensor(masks), "positions": torch.tensor([positions] * s["case"]["axes"])}


def _exact_tree(s):
    c = s["case"]
    if work(c)["flops"] > 4e12:
        return None
    H, G, P = c["hkv"], c["hq"] // c["hkv"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (q, n) in enumerate(_lengths(c)):
        ids = s["table"][b, :-(-n // P)].long()
        bits = torch.stack([(s["masks"][at:at + q, i // 32] >> (i % 32)) & 1 for i in range(q)], 1).bool()
        bits &= torch.ones_like(bits).tril()
        seen = torch.cat([torch.ones(q, n - q, dtype=torch.bool, device=out.device), bits], 1)
        for h in range(H):
            k, v = (s[x][ids, :, h].flatten(0, 1)[:n].double() * d for x, d in (("k", c["kd"]), ("v", c["vd"])))
            for g in range(h * G, (h + 1) * G):
                x = s["q"][at:at + q, g].double() @ k.T / 16
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                w = torch.softmax(x, -1)
                out[at:at + q, g] = torch.where(seen.any(1, keepdim=True), w, torch.zeros_like(w)) @ v
        at += q
    return {"out": out}


def _exact_e4m3(x):
    """The nearest e4m3 value (4 significant bits, 2^-9 at least, a tie to the even one), at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_keep(s):
    c = s["case"]
    P = c["page"]
    got = {"k": s["k"].double(), "v": s["v"].double()}
    lens = []
    at = 0
    for b, (q, n) in enumerate(_lengths(c)):
        ids = s["table"][b].tolist()
        kept = s["kept"][b, :int(s["num"][b])].tolist()
        places = list(range(n - q, n)) + list(range(n - q, n - q + len(kept)))  # every new token where it was drafted, then the kept ones
        tokens = list(range(q)) + kept
        final = dict(zip(places, tokens))
        page, slot = ([ids[x // P] for x in final], [x % P for x in final])
        tok = [at + x for x in final.values()]
        for name, descale in (("k", c["kd"]), ("v", c["vd"])):
            got[name][page, slot] = _exact_e4m3(s[name + "_new"][tok].double() / descale)
        lens.append(n - q + len(kept))
        at += q
    return {**got, "lens": torch.tensor(lens)}


def _exact_prompt(s):
    c = s["case"]
    G = c["hq"] // c["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=out.device)
    at = 0
    for n, _ in _lengths(c):
        for g in range(c["hq"]):
            k, v = (s[x][at:at + n, g // G].double() for x in ("k", "v"))
            for t0 in range(0, n, 2048):  # rows in runs, for their scores' memory
                t1 = min(n, t0 + 2048)
                x = s["q"][at + t0:at + t1, g].double() @ k[:t1].T / 16
                x += torch.full_like(x, -math.inf).triu(t0 + 1)
                lse[at + t0:at + t1, g] = torch.logsumexp(x, -1)
                out[at + t0:at + t1, g] = torch.softmax(x, -1) @ v[:t1]
        at += n
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
