"""Inputs and checks of the tests of block tables, token trees and prompts."""
import random

import numpy as np
import torch

import workloads as wl
from oracle import step

D = wl.HEAD_DIM


def requests(seed, S, P, W, q_hi=5, ctx_hi=400, ended=0.1, pad=0.1, admit=0.2, spare=True, short=0):
    """Lists of a valid step's inputs; `short`: so many pages fewer are free than are needed."""
    r = random.Random(seed)
    R = S + 3
    rows = r.sample(range(R), S)
    q, ctx, held, need = [], [], [], 0
    for s in range(S):
        kind = r.random()
        c, n = r.randint(0, ctx_hi), r.randint(0, q_hi)
        if kind < pad:
            rows[s], c, n = -1, 0, 0
        elif kind < pad + ended:
            n = -1
        elif kind < pad + ended + admit:
            c, n = 0, r.randint(1, ctx_hi)
        q.append(n)
        ctx.append(c)
        h = -(-c // P) + (r.randint(0, 1) if spare and rows[s] >= 0 and -(-c // P) < W else 0)
        held.append(h)
        if n >= 0 and rows[s] >= 0:
            need += max(0, -(-(c + n) // P) - h)
        elif rows[s] >= 0:
            need -= h
    F = sum(held) + max(need, 0) + 7
    ids = r.sample(range(F), F)
    pages, counts = [[-1] * W for _ in range(R)], [0] * R
    for s in range(S):
        if rows[s] >= 0:
            counts[rows[s]] = held[s]
            pages[rows[s]][:held[s]] = ids[:held[s]]
            del ids[:held[s]]
    top = max(0, min(len(ids), max(need, 0)) - short) if short else len(ids)
    free = ids[:top] + [-7] * (F - top)
    return dict(q_lens=q, ctx_lens=ctx, rows=rows, page_size=P, pages=pages, counts=counts, free=free, num_free=top)


def run_tables(x, W, T, in_place=False, dev="cuda"):
    import paged_gqa_gb300 as pg
    t = {n: torch.tensor(x[n] if n != "num_free" else [x[n]], dtype=torch.int32, device=dev)
         for n in ("q_lens", "ctx_lens", "rows", "pages", "counts", "free", "num_free")}
    S = len(x["q_lens"])
    new = lambda *shape: torch.full(shape, -99, dtype=torch.int32, device=dev)  # noqa: E731
    table, lens, qsl, slots = new(S, W), new(S), new(S + 1), new(T)
    co, no = (None, None) if in_place else (new(t["counts"].numel()), new(1))
    pg.paged_gqa_build_tables(t["q_lens"], t["ctx_lens"], t["rows"], x["page_size"], t["pages"], t["counts"], t["free"], t["num_free"],
                              table, lens, qsl, slots, co, no)
    status = pg.paged_gqa_check_device_errors()
    if not in_place:  # the inputs stay
        assert t["counts"].tolist() == x["counts"] and t["num_free"].tolist() == [x["num_free"]]
    got = dict(table=table, lens=lens, qsl=qsl, slots=slots, pages=t["pages"], counts=t["counts"] if in_place else co, free=t["free"],
               num_free=t["num_free"] if in_place else no)
    return {n: y.tolist() for n, y in got.items()}, status


def check_tables(x, W, T, in_place=False):
    ref = {n: ([list(y) for y in v] if n == "pages" else list(v) if isinstance(v, list) else v) for n, v in x.items()}
    got, status = run_tables(x, W, T, in_place)
    want = step.build_tables(**ref, width=W, tokens=T)
    assert status == (-5 if want.pop("bad") else 0)
    for name in want:
        assert got[name] == want[name], name


def parents(r, n):
    return [-1 if t == 0 or r.random() < 0.1 else r.randint(max(0, t - 6), t - 1) if r.random() < 0.5 else r.randrange(t) for t in range(n)]


class Tree:
    """A tree step on a paged cache; poisoned slots and pages hold NaN, the cache's tokens N(0, 1)."""

    def __init__(self, seqs, hq, hkv, P, cache="e4m3", seed=0, words=None, masks="tree", dev="cuda"):
        r, gen = random.Random(seed), torch.Generator().manual_seed(seed)
        self.seqs, self.hq, self.hkv, self.P, self.cache = seqs, hq, hkv, P, cache
        T = self.T = sum(n for n, _ in seqs)
        self.words = words or max(1, -(-max(n for n, _ in seqs) // 32))
        self.parents = [p for n, _ in seqs for p in parents(r, n)]
        self.qsl = [0]
        for n, _ in seqs:
            self.qsl.append(self.qsl[-1] + n)
        self.lens = [L for _, L in seqs]
        if masks == "tree":
            self.masks = step.tree_masks(self.parents, self.lens, self.qsl, self.words)[0]
        elif masks == "none":
            self.masks = [[0] * self.words for _ in range(T)]
        elif masks == "all":
            self.masks = [[-1] * self.words for _ in range(T)]
        else:
            self.masks = [[r.randint(-2 ** 31, 2 ** 31 - 1) & r.choice([0, -1, 0x55555555]) for _ in range(self.words)] for _ in range(T)]
        need = [-(-L // P) for _, L in seqs]
        NB, W = sum(need) + 2, max(need) + 1
        order = torch.randperm(NB, generator=gen).tolist()
        table = [[-1] * W for _ in seqs]
        kind = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
        self.k_descale, self.v_descale = (1.0, 1.0) if cache == "bf16" else (0.25, 0.5)
        kv = [torch.full((NB, P, hkv, D), float("nan")) for _ in range(2)]
        at = 0
        for s, (_, L) in enumerate(seqs):
            table[s][:need[s]] = order[at:at + need[s]]
            at += need[s]
            for c, d in zip(kv, (self.k_descale, self.v_descale)):
                x = torch.randn(need[s] * P, hkv, D, generator=gen) / d
                x[L:] = float("nan")
                c[table[s][:need[s]]] = x.view(need[s], P, hkv, D)
        self.k, self.v = (c.to(kind).to(dev) for c in kv)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        self.table, self.lens_t, self.qsl_t, self.masks_t, self.parents_t = i32(table), i32(self.lens), i32(self.qsl), i32(self.masks), i32(self.parents)
        self.q = torch.randn(T, hq, D, generator=gen).bfloat16().to(dev)
        self.scale = 1 / 16

    def args(self, **over):
        a = dict(q=self.q, k=self.k, v=self.v, bt=self.table, sl=self.lens_t, qsl=self.qsl_t, masks=self.masks_t)
        a.update(over)
        return list(a.values()) + [self.k_descale, self.v_descale, self.scale]

    def run(self, out=None, check=True, **over):
        import paged_gqa_gb300 as pg
        out = torch.full_like(self.q, float("nan")) if out is None else out
        pg.paged_gqa_attn_tree(*self.args(**over), out)
        if check:
            assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()
        return out

    def reference(self):
        ref = np.zeros((self.T, self.hq, D))
        q, k, v = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        G = self.hq // self.hkv
        for s, (n, L) in enumerate(self.seqs):
            q0 = self.qsl[s]
            ids = self.table[s, :-(-L // self.P)].tolist()
            seen = step.tree_seen(self.masks[q0:q0 + n], n, L)
            for h in range(self.hkv):
                ks, vs = (x[ids, :, h].reshape(-1, D)[:L] * d for x, d in ((k, self.k_descale), (v, self.v_descale)))
                for g in range(h * G, (h + 1) * G):
                    ref[q0:q0 + n, g] = step.attention(q[q0:q0 + n, g], ks, vs, seen, self.scale)[0]
        return ref


def compare(got, ref, what=""):
    """The bar of the paged calls (1e-2 and 5e-3 relative in the 2-norm), with the output's own rounding beside it: a
    row that sees one key is that key's V, |V| reaches 4.4 among the N(0, 1) values here, and half a bf16 step
    of it is 4.4 * 2^-8 = 1.7e-2 by itself. So a value may be off by 1e-2 + 2^-8 |value|."""
    g = got.detach().double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(g).all(), what
    diff = np.abs(g - ref)
    worst = (diff - 2.0 ** -8 * np.abs(ref)).max(initial=0.0)
    rel = np.linalg.norm(diff) / (np.linalg.norm(ref) or 1.0)
    assert worst <= 1e-2 and rel <= 5e-3, f"{what}: {worst:.3e} over the rounding, relative {rel:.3e}"


U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative to the value


class Prompt:
    def __init__(self, lens, hq, hkv, dtype=torch.bfloat16, seed=0, fused=True, behind=0, dev="cuda", scale=1 / 16, size=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.dtype, self.scale = lens, hq, hkv, dtype, scale
        T = self.T = sum(lens) + behind
        x = torch.randn(T, hq + 2 * hkv, D, generator=gen) * size
        if behind:
            x[T - behind:] = float("nan")  # rows of no prompt
        x = x.to(dtype).to(dev)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not fused:
            self.q, self.k, self.v = (y.contiguous() for y in (self.q, self.k, self.v))
        self.qsl = [0]
        for n in lens:
            self.qsl.append(self.qsl[-1] + n)
        self.qsl_t = torch.tensor(self.qsl, dtype=torch.int32, device=dev)

    def run(self, lse=True, check=True, out=None):
        import paged_gqa_gb300 as pg
        out = torch.full(self.q.shape, float("nan"), dtype=self.dtype, device=self.q.device) if out is None else out
        ls = torch.full(self.q.shape[:2], float("nan"), device=self.q.device) if lse else None
        pg.paged_gqa_attn_prompt(self.q, self.k, self.v, self.qsl_t, self.scale, out, ls)
        if check:
            assert pg.paged_gqa_check_device_errors() == 0, pg.paged_gqa_last_error()
        return out, ls

    def check(self, out, lse, rows=None):
        """Each value against the definition in 64 bits. What may be off, relative to sum w |v|: P's rounding
        (u), the scores' (256 fp32 additions: 2^-15 of sum |q||k| scale, in numerator and denominator), the sums
        over n keys (n 2^-23), the exponentials (2^-20); the output's rounding (u |o|); f16 values of P below
        2^-14 (2^-25 of a reference of at least 1, n of them). rows: {sequence: tokens to look at}."""
        u, G = U[self.dtype], self.hq // self.hkv
        q, k, v = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        o, ls = out.double().cpu().numpy(), lse.double().cpu().numpy() if lse is not None else None
        for s, n in enumerate(self.lens):
            if n == 0 or (rows is not None and s not in rows):
                continue
            at = self.qsl[s]
            t = np.arange(n) if rows is None else np.array(rows[s])
            seen = np.arange(n) <= t[:, None]
            for g in range(self.hq):
                kk, vv = k[at:at + n, g // G], v[at:at + n, g // G]
                want, mag, l, size = step.attention(q[at + t, g], kk, vv, seen, self.scale)
                ds = (size * 2.0 ** -15 + 2.0 ** -20)[:, None]
                tol = mag * (u + 2 * ds + n * 2.0 ** -23) + u * np.abs(want)
                if self.dtype is torch.float16:
                    tol += n * 2.0 ** -25 * np.abs(vv).max()
                got = o[at + t, g]
                assert np.isfinite(got).all(), (s, g)
                worst = np.max(np.abs(got - want) / tol)
                assert worst <= 1.0, (s, g, worst)
                if ls is not None:
                    bound = ds[:, 0] + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(l)
                    worst = np.max(np.abs(ls[at + t, g] - l) / bound)
                    assert worst <= 1.0, (s, g, worst)
