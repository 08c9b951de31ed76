"""The 4-bit paged KV cache and the rotary positions in front of it: the cases they are measured on.

`run` with `own` false computes each operator from elementary torch operations in float32 (float64 for
angles); with `own` true it makes the calls of paged_gqa_gb300. Cache layout (include/paged_gqa.h): a
(token, kv head) row of 256 values is 128 bytes of e2m1 codes (byte i: d = 2i in the low nibble, 2i + 1 in
the high one) and 16 e4m3 scales, one per 16 values; value = code * scale * descale. Caches are uint8
[pages, kv heads, P, 144]: K rows token by token, V in blocks of 16 tokens, each [128 bytes][16 tokens] of
codes and then [16 groups][16 tokens] of scales.
"""
import math

import torch

own = False

D = 256
ROW = 144
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases --

def listed():
    return [
        # attention: one sequence, one new token (the smallest call: its latency is what counts)
        dict(name="attn_one_token", op="attn", seqs=1, q_lo=1, q_hi=1, l_lo=600, l_hi=600, hq=16, hkv=1, page=16, chunks=0, chunk_q=0),
        # a batch that decodes one token per sequence, 64-token pages
        dict(name="attn_decode", op="attn", seqs=32, q_lo=1, q_hi=1, l_lo=2048, l_hi=16384, hq=8, hkv=1, page=64, chunks=0, chunk_q=0),
        # speculative verify: 4 tokens per sequence, ragged contexts, 16-token pages
        dict(name="attn_verify", op="attn", seqs=64, q_lo=4, q_hi=4, l_lo=1024, l_hi=32768, hq=16, hkv=1, page=16, chunks=0, chunk_q=0),
        # the widest batch, two kv heads
        dict(name="attn_verify_wide", op="attn", seqs=256, q_lo=2, q_hi=4, l_lo=8192, l_hi=8192, hq=32, hkv=2, page=16, chunks=0, chunk_q=0),
        # decoding and prefill chunks of odd lengths in one call
        dict(name="attn_mixed", op="attn", seqs=15, q_lo=1, q_hi=4, l_lo=777, l_hi=9001, hq=24, hkv=2, page=64, chunks=3, chunk_q=611),
        # a prefill chunk on a long context: bound by the matrix products
        dict(name="attn_prefill", op="attn", seqs=1, q_lo=8192, q_hi=8192, l_lo=32768, l_hi=32768, hq=8, hkv=1, page=64, chunks=0, chunk_q=0),
        # rotary of one verify step's tokens (64 sequences x 4), a quarter of the head rotated
        dict(name="rope_verify", op="rope", tokens=256, hq=16, hkv=1, rot=64, axes=3, interleaved=True, adjacent=False, far=40000),
        # rotary of a prefill batch, the whole head rotated, positions far out
        dict(name="rope_prefill", op="rope", tokens=16384, hq=24, hkv=2, rot=256, axes=3, interleaved=False, adjacent=True, far=1000000),
        # writing one verify step's tokens and reading back what the cache holds of them
        dict(name="write_verify", op="write", seqs=64, q_lo=4, q_hi=4, l_lo=1024, l_hi=32768, hkv=1, page=16),
        # writing prefill chunks of odd lengths at odd offsets
        dict(name="write_chunks", op="write", seqs=8, q_lo=8001, q_hi=8192, l_lo=8192, l_hi=24576, hkv=2, page=64),
        # reading the last tokens of a few short sequences
        dict(name="read_short", op="read", seqs=5, q_lo=33, q_hi=330, l_lo=400, l_hi=1500, hkv=1, page=16),
        # reading whole prefixes, to move them to another cache
        dict(name="read_prefix", op="read", seqs=6, q_lo=4097, q_hi=16384, l_lo=16384, l_hi=16384, hkv=2, page=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "rope", "write", "read"])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        hq, hkv = rng.choice([(8, 1), (16, 1), (32, 2), (24, 2), (6, 1), (5, 5)])
        return dict(op="rope", tokens=_log_int(rng, 1, 12000), hq=hq, hkv=hkv, rot=rng.choice([32, 64, 96, 128, 192, 256]),
                    axes=rng.choice([1, 2, 3, 4]), interleaved=rng.random() < 0.5, adjacent=rng.random() < 0.5,
                    far=_log_int(rng, 100, 2000000))
    if op in ("write", "read"):
        seqs = _log_int(rng, 1, 64)
        q_hi = _log_int(rng, 1, max(2, 48000 // seqs))
        l_hi = q_hi + _log_int(rng, 1, 16384)
        q_lo = rng.randint(1, q_hi)
        return dict(op=op, seqs=seqs, q_lo=q_lo, q_hi=q_hi, l_lo=rng.randint(q_hi, l_hi), l_hi=l_hi, hkv=rng.choice([1, 2, 4]) if seqs * q_hi < 10000 else 1, page=page)
    hq, hkv = rng.choice([(8, 1), (16, 1), (32, 2), (24, 2), (6, 1), (12, 1), (8, 4), (3, 1)])
    kind = rng.choice(["decode", "verify", "mixed", "prefill"])
    if kind == "prefill":
        seqs, q_hi = rng.choice([1, 1, 2, 3]), _log_int(rng, 65, 3500)
        l_hi = q_hi + _log_int(rng, 1, 14000)
        return dict(op="attn", seqs=seqs, q_lo=rng.randint(max(1, q_hi // 2), q_hi), q_hi=q_hi, l_lo=rng.randint(q_hi, l_hi), l_hi=l_hi,
                    hq=8, hkv=rng.choice([1, 2]), page=page, chunks=0, chunk_q=0)
    if kind == "mixed":
        l_hi = _log_int(rng, 600, 8000)
        return dict(op="attn", seqs=rng.randint(1, 12), q_lo=1, q_hi=rng.randint(1, 4), l_lo=rng.randint(500, l_hi), l_hi=l_hi, hq=hq, hkv=hkv,
                    page=page, chunks=rng.randint(1, 3), chunk_q=rng.randint(17, 400))
    q_hi = 1 if kind == "decode" else rng.randint(2, 4)
    seqs = _log_int(rng, 1, 128)
    l_hi = _log_int(rng, 5, min(40000, 1000000 // seqs))
    return dict(op="attn", seqs=seqs, q_lo=1, q_hi=q_hi, l_lo=rng.randint(min(4, l_hi), l_hi), l_hi=l_hi, hq=hq, hkv=hkv, page=page, chunks=0, chunk_q=0)


def _lengths(case, seed=None):
    """[(q_len, L)] of the batch: the same for every seed, so that `work` can count them."""
    gen = torch.Generator().manual_seed(20 + case["seqs"] + 7 * case["l_hi"] + 13 * case["q_hi"])

    def between(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=gen).tolist()

    seqs = list(zip(between(case["q_lo"], case["q_hi"], case["seqs"]), between(case["l_lo"], case["l_hi"], case["seqs"])))
    for i in range(case.get("chunks", 0)):  # prefill chunks among the decoding sequences
        n = max(1, case["chunk_q"] - 37 * i)
        seqs.insert(3 * i + 1, (n, max(n, case["l_hi"] - 101 * i)))
    return [(min(q, n), n) for q, n in seqs]


def work(case):
    if case["op"] == "rope":
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": rows * D * 2 * 2 + case["axes"] * case["tokens"] * 4 + case["rot"] * 2, "flops": rows * case["rot"] // 2 * 6}
    seqs = _lengths(case)
    tables = sum(-(-n // case["page"]) for _, n in seqs) * 4 + len(seqs) * 8
    T = sum(q for q, _ in seqs)
    if case["op"] == "attn":
        pairs = sum(q * (n - q + 1) + q * (q - 1) // 2 for q, n in seqs)
        return {"bytes": sum(n for _, n in seqs) * case["hkv"] * 2 * ROW + T * case["hq"] * D * 4 + tables, "flops": 4 * D * case["hq"] * pairs}
    rows = T * case["hkv"]
    once = rows * (2 * D * 2 + 2 * ROW) + T * 4  # bf16 rows on one side, codes and scales on the other
    return {"bytes": 2 * once if case["op"] == "write" else once, "flops": rows * 2 * D * 4}


# ----------------------------------------------------------------------------------------- inputs --

def _quantise(x, descale):
    """x [..., 256] -> (bytes [..., 128], scales [..., 16] as e4m3 bits), float32 steps."""
    y = x.float() * (torch.ones((), device=x.device) / torch.tensor(descale, dtype=torch.float32, device=x.device))
    g = y.unflatten(-1, (16, 16))
    s8 = (g.abs().amax(-1) * torch.tensor(1.0 / 6.0, dtype=torch.float32, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    r = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    z = g * r.unsqueeze(-1)
    a = z.abs()
    # round to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, a tie to the even code
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    c = torch.where(torch.signbit(z), m + 8, m).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], s8.view(torch.uint8)


def _pack_k(codes, scales):
    return torch.cat([codes, scales], -1)


def _pack_v(codes, scales):
    """[..., P, 128] and [..., P, 16] -> [..., P, 144] in blocks of 16 tokens."""
    P = codes.shape[-2]
    c = codes.unflatten(-2, (P // 16, 16)).transpose(-1, -2).flatten(-2)
    s = scales.unflatten(-2, (P // 16, 16)).transpose(-1, -2).flatten(-2)
    return torch.cat([c, s], -1).flatten(-2).unflatten(-1, (P, ROW))


def _cache(case, seqs, gen, dev):
    """Two filled caches with their pages in random order; slots that no sequence holds are 0xFF (NaN scales)."""
    P, H = case["page"], case["hkv"]
    need = [-(-n // P) for _, n in seqs]
    NB, W = sum(need) + 3, max(need) + 1
    order = torch.randperm(NB, generator=gen, device=dev)
    table = torch.full((len(seqs), W), -1, dtype=torch.int32, device=dev)
    held = torch.zeros(NB, P, dtype=torch.bool, device=dev)
    at = 0
    for i, (_, n) in enumerate(seqs):
        mine = order[at:at + need[i]]
        table[i, :need[i]] = mine.int()
        held[mine] = (torch.arange(need[i] * P, device=dev) < n).view(-1, P)
        at += need[i]
    caches = []
    for descale, pack in ((case["kd"], _pack_k), (case["vd"], _pack_v)):
        buf = torch.empty(NB, H, P, ROW, dtype=torch.uint8, device=dev)
        # some channels of K are larger than others, as in trained models
        size = torch.exp(0.5 * torch.randn(D, generator=gen, device=dev)) if pack is _pack_k else torch.ones(D, device=dev)
        step = max(1, (1 << 26) // (H * P * D))
        for b in range(0, NB, step):
            x = torch.randn(min(step, NB - b), H, P, D, generator=gen, device=dev) * size
            codes, scales = _quantise(x, descale)
            out = ~held[b:b + step, None, :, None]
            buf[b:b + step] = pack(codes.masked_fill(out, 255), scales.masked_fill(out, 255))
        caches.append(buf)
    return caches[0], caches[1], table


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "rope":
        T, hq, hkv, R, A = (case[k] for k in ("tokens", "hq", "hkv", "rot", "axes"))
        qkv = torch.randn(T, hq + 2 * hkv, D, generator=gen, device=dev).bfloat16()  # one projection's output
        pos = torch.randint(0, case["far"], (A, T), generator=gen, device=dev, dtype=torch.int32)
        inv = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)).float()
        part = R // 2 // A
        sections = [R // 2 - part * (A - 1)] + [part] * (A - 1)
        return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], pos=pos, inv=inv, sections=sections,
                    q_out=torch.empty(T, hq, D, dtype=torch.bfloat16, device=dev), k_out=torch.empty(T, hkv, D, dtype=torch.bfloat16, device=dev))
    seqs = _lengths(case)
    # a per-tensor descale near amax / (6 * 448), another for every seed
    kd, vd = (torch.rand(2, generator=torch.Generator().manual_seed(seed)) * 0.002 + 0.002).tolist()
    case = dict(case, kd=kd, vd=vd)
    k, v, table = _cache(case, seqs, gen, dev)
    T = sum(q for q, _ in seqs)
    qsl = torch.tensor([0] + [q for q, _ in seqs], device=dev).cumsum(0).int()
    lens = torch.tensor([n for _, n in seqs], dtype=torch.int32, device=dev)
    s = dict(case=case, k=k, v=v, table=table, qsl=qsl, lens=lens, q_max=max(q for q, _ in seqs))
    if case["op"] == "attn":
        s["q"] = torch.randn(T, case["hq"], D, generator=gen, device=dev).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        return s
    if case["op"] == "write":
        s["k_new"], s["v_new"] = (torch.randn(T, case["hkv"], D, generator=gen, device=dev).bfloat16() for _ in range(2))
    s["k_out"], s["v_out"] = (torch.empty(T, case["hkv"], D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    return s


# -------------------------------------------------------------------------------------- the passes --

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "rope":
        return _plain_rope(s)
    if op == "attn":
        return _plain_attn(s)
    if op == "write":
        _plain_write(s)
    return _plain_read(s)


def _own(s):
    import paged_gqa_gb300 as pg
    c = s["case"]
    if c["op"] == "rope":
        pg.paged_gqa_rope(s["q"], s["k"], s["pos"], s["inv"], s["sections"], s["q_out"], s["k_out"],
                          interleaved=c["interleaved"], adjacent=c["adjacent"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "attn":
        pg.paged_gqa_attn_fp4(s["q"], s["k"], s["v"], s["table"], s["lens"], s["qsl"], c["kd"], c["vd"], 1 / 16, s["out"])
        return {"out": s["out"]}
    if c["op"] == "write":
        pg.paged_gqa_cache_write_fp4(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], s["qsl"], c["kd"], c["vd"])
    pg.paged_gqa_cache_read_fp4(s["k"], s["v"], s["table"], s["lens"], s["qsl"], c["kd"], c["vd"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _axis_of(sections, interleaved, dev):
    """The axis of each frequency."""
    n, A = sum(sections), len(sections)
    i = torch.arange(n, device=dev)
    if interleaved:  # axis a has every A-th frequency until it has its number; the first axis has the rest
        a = i % A
        return torch.where(i < A * torch.tensor(sections, device=dev)[a], a, torch.zeros_like(a))
    return torch.repeat_interleave(torch.arange(A, device=dev), torch.tensor(sections, device=dev), output_size=n)


def _plain_rope(s):
    c = s["case"]
    R = c["rot"]
    pos = s["pos"].double()[_axis_of(s["sections"], c["interleaved"], s["pos"].device)].t()
    ang = pos * s["inv"].double()
    cos, sin = ang.cos().float().unsqueeze(1), ang.sin().float().unsqueeze(1)

    def turned(x):
        y = x.float().clone()
        a, b = (slice(0, R, 2), slice(1, R, 2)) if c["adjacent"] else (slice(0, R // 2), slice(R // 2, R))
        u, w = y[..., a].clone(), y[..., b].clone()
        y[..., a] = u * cos - w * sin
        y[..., b] = w * cos + u * sin
        return y.bfloat16()

    return {"q": turned(s["q"]), "k": turned(s["k"])}


def _values(codes, scales):
    """Code bytes [..., 128] and scale bytes [..., 16] -> float32 [..., 256]."""
    lut = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    both = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], -1)  # byte -> its two values
    x = both.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], 16, 16)
    return (x * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _places(s):
    """Each new token's page, slot and sequence."""
    c = s["case"]
    T = s["k_out"].shape[0]
    t = torch.arange(T, device=s["qsl"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["qsl"], t, right=True) - 1
    pos = s["lens"][seq] - (s["qsl"][seq + 1] - t)
    return s["table"][seq, (pos // c["page"]).long()].long(), (pos % c["page"]).long()


def _v_parts(v):
    """Views of a V cache: codes [NB, H, blocks, 128, 16 tokens] and scales [NB, H, blocks, 16, 16 tokens]."""
    b = v.flatten(-2).unflatten(-1, (-1, 16 * ROW))
    return b[..., :2048].unflatten(-1, (128, 16)), b[..., 2048:].unflatten(-1, (16, 16))


def _plain_write(s):
    c = s["case"]
    page, slot = _places(s)
    h = torch.arange(c["hkv"], device=page.device)
    page, slot = page.unsqueeze(1), slot.unsqueeze(1)
    s["k"][page, h, slot] = _pack_k(*_quantise(s["k_new"], c["kd"]))
    codes, scales = _quantise(s["v_new"], c["vd"])
    vc, vs = _v_parts(s["v"])
    vc[page, h, slot // 16, :, slot % 16] = codes
    vs[page, h, slot // 16, :, slot % 16] = scales


def _plain_read(s):
    c = s["case"]
    page, slot = _places(s)
    h = torch.arange(c["hkv"], device=page.device)
    page, slot = page.unsqueeze(1), slot.unsqueeze(1)
    rows = s["k"][page, h, slot]
    vc, vs = _v_parts(s["v"])
    k = _values(rows[..., :128], rows[..., 128:].contiguous())
    v = _values(vc[page, h, slot // 16, :, slot % 16], vs[page, h, slot // 16, :, slot % 16])
    return {"k": (k * c["kd"]).bfloat16(), "v": (v * c["vd"]).bfloat16()}


def _plain_attn(s):
    c = s["case"]
    H, G, P = c["hkv"], c["hq"] // c["hkv"], c["page"]
    dev = s["q"].device
    pages = s["table"].clamp(min=0).long()
    S, W = pages.shape
    j = torch.arange(W * P, device=dev)
    held = (j < s["lens"].unsqueeze(1))[:, None, :, None]
    rows = s["k"][pages]  # [S, W, H, P, 144]
    k = _values(rows[..., :128], rows[..., 128:].contiguous()).transpose(1, 2).flatten(2, 3)
    k = k.masked_fill(~held, 0.0)
    del rows
    vc, vs = _v_parts(s["v"][pages])
    v = _values(vc.transpose(-1, -2), vs.transpose(-1, -2).contiguous()).flatten(3, 4).transpose(1, 2).flatten(2, 3)
    v = v.masked_fill(~held, 0.0)
    # the new tokens of each sequence, padded to the longest; row t of a sequence sees keys 0 .. L - q_len + t
    t = torch.arange(s["q_max"], device=dev)
    qn = (s["qsl"][1:] - s["qsl"][:-1]).long()
    real = t < qn.unsqueeze(1)
    token = (s["qsl"][:-1].long().unsqueeze(1) + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][token].float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [S, H, q_max * G, 256]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(c["kd"] / 16)
    last = (s["lens"].long() - qn).unsqueeze(1) + t
    seen = ((j <= last.unsqueeze(-1)) & real.unsqueeze(-1)).repeat_interleave(G, 1).unsqueeze(1)
    p.masked_fill_(~seen, -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30) * c["vd"]
    o = o.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).flatten(2, 3).bfloat16()
    out = torch.zeros_like(s["q"])
    out[token[real]] = o[real]
    return {"out": out}


# ------------------------------------------------------------------- the definition, in 64 bits --

def _exact_row(codes, scales, descale):
    """float64 values from the bits: sign, exponent and fraction of each code and scale."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int64)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, m / 2, torch.ldexp(1 + m / 2, e - 1))
    x = torch.where(n >= 8, -mag, mag)
    b = scales.to(torch.int64)
    se, sm = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(se == 0, sm / 512, torch.ldexp(1 + sm / 8, se - 7))
    sc = torch.where((b & 127) == 127, torch.full_like(sc, math.nan), torch.where(b >= 128, -sc, sc))
    return x * sc.repeat_interleave(16, -1) * descale


def _exact_kv(s, i, n, head):
    """The first n keys and values of sequence i in float64."""
    c = s["case"]
    P = c["page"]
    page = s["table"][i, :-(-n // P)].long()
    k = s["k"][page, head].reshape(-1, ROW)[:n]
    v = s["v"][page, head].reshape(-1, 16 * ROW)
    codes = v[:, :2048].reshape(-1, 128, 16).permute(0, 2, 1).reshape(-1, 128)[:n]
    scales = v[:, 2048:].reshape(-1, 16, 16).permute(0, 2, 1).reshape(-1, 16)[:n]
    return _exact_row(k[:, :128], k[:, 128:], c["kd"]), _exact_row(codes, scales, c["vd"])


def _exact_stored(x, descale):
    """What a cache holds of x [N, 256], float64: the nearest e4m3 scale to the sixth of each group's largest
    value, the nearest e2m1 code to each value in its units (a tie to the even code)."""
    y = (x.double() / descale).reshape(-1, 16, 16)
    sc = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(sc.clamp(min=2.0 ** -6))) - 3)
    sc = torch.round(sc / step) * step  # to 3 fraction bits, 2^-9 at least; torch.round ties to even
    z = torch.where(sc > 0, y / sc, torch.zeros_like(y)).clamp(-6, 6)
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=1.0))) - 1)
    return (torch.round(z / step) * step * sc).reshape(-1, D) * descale


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        R, n = c["rot"], c["rot"] // 2
        axis = []
        for a, count in enumerate(s["sections"]):
            axis += [a] * count
        if c["interleaved"]:
            left, axis = list(s["sections"]), []
            for i in range(n):
                a = i % c["axes"]
                a = a if i // c["axes"] < s["sections"][a] else 0
                axis.append(a)
        got = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            for i in range(n):
                ang = s["pos"][axis[i]].double() * s["inv"][i].double()
                turn = torch.polar(torch.ones_like(ang), ang).unsqueeze(1)
                a, b = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + n)
                z = torch.complex(x[..., a], x[..., b]) * turn
                y[..., a], y[..., b] = z.real, z.imag
            got[name] = y
        return got
    seqs = _lengths(c)
    H = c["hkv"]
    if c["op"] == "write":
        return {"k": _exact_stored(s["k_new"].reshape(-1, D), c["kd"]).reshape(-1, H, D), "v": _exact_stored(s["v_new"].reshape(-1, D), c["vd"]).reshape(-1, H, D)}
    if c["op"] == "read":
        got = {"k": [], "v": []}
        for i, (q, n) in enumerate(seqs):
            kv = [_exact_kv(s, i, n, h) for h in range(H)]
            got["k"].append(torch.stack([x[0][n - q:] for x in kv], 1))
            got["v"].append(torch.stack([x[1][n - q:] for x in kv], 1))
        return {name: torch.cat(x) for name, x in got.items()}
    if work(c)["flops"] > 6e12:
        return None
    G = c["hq"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for i, (q, n) in enumerate(seqs):
        for h in range(H):
            k, v = _exact_kv(s, i, n, h)
            for t0 in range(0, q, 512):  # rows in runs, for their scores' memory
                t1 = min(q, t0 + 512)
                rows = s["q"][at + t0:at + t1, h * G:(h + 1) * G].double().reshape(-1, D)
                limit = torch.arange(n - q + t0, n - q + t1, device=rows.device).repeat_interleave(G)
                x = rows @ k.T / 16
                x = torch.where(torch.arange(n, device=rows.device) <= limit.unsqueeze(1), x, torch.full_like(x, -math.inf))
                out[at + t0:at + t1, h * G:(h + 1) * G] = (torch.softmax(x, -1) @ v).reshape(t1 - t0, G, D)
        at += q
    return {"out": out}
