"""What surrounds the attention of a step, and attention by masks and over prompts, from their definitions.

Plain loops and float64; shares nothing with the library. Request by request, token by token.
"""
from __future__ import annotations

import numpy as np

INT_MAX = 2 ** 31 - 1


def build_tables(q_lens, ctx_lens, rows, page_size, pages, counts, free, num_free, width, tokens):
    """The step's tables; pages and free are changed in place (lists). Returns a dict; 'bad' tells of a flag."""
    S, R, Wp, F = len(q_lens), len(pages), len(pages[0]) if pages else 0, len(free)
    counts = list(counts)
    top, bad = num_free, False
    if not 0 <= top <= F:
        bad, top = True, min(max(top, 0), F)
    valid, owner = [], {}
    for s in range(S):
        r = rows[s]
        ok = 0 <= r < R and 0 <= counts[r] <= Wp
        if ok and r in owner:
            ok = False
        elif ok:
            owner[r] = s
        valid.append(ok)
        bad |= not ok and r != -1
    full = False  # a stack that would overflow takes nothing more
    for s in range(S):
        if valid[s] and q_lens[s] == -1:
            n = counts[rows[s]]
            if n and (full or top + n > F):
                bad = full = True
                continue
            free[top:top + n] = pages[rows[s]][:n]
            top += n
            counts[rows[s]] = 0
    table, lens, qsl, slots = [], [], [0], []
    dry = False
    for s in range(S):
        q, r = q_lens[s], rows[s]
        row, length = [-1] * width, 0
        new = max(q, 0) if r != -1 else 0
        bad |= r == -1 and q > 0 or (r != -1 and q < -1)
        got = [-1] * new
        if valid[s] and q >= 0:
            length = ctx_lens[s] + q
            need = -(-length // page_size)
            take = max(0, need - counts[r])
            if ctx_lens[s] < 0 or length > INT_MAX or need > min(width, Wp):
                length, bad = 0, True
            elif take and (dry or take > top):
                length, bad, dry = 0, True, True
            else:
                for _ in range(take):
                    top -= 1
                    pages[r][counts[r]] = free[top]
                    counts[r] += 1
                row[:need] = pages[r][:need]
                for t in range(q):
                    pos = ctx_lens[s] + t
                    slot = pages[r][pos // page_size] * page_size + pos % page_size
                    ok = pages[r][pos // page_size] >= 0 and slot <= INT_MAX
                    bad |= not ok
                    got[t] = slot if ok else -1
        table.append(row)
        lens.append(length)
        qsl.append(qsl[-1] + new)
        slots += got
    bad |= len(slots) > tokens
    return dict(table=table, lens=lens, qsl=qsl, slots=(slots + [-1] * tokens)[:tokens], pages=pages, counts=counts, free=free,
                num_free=[top], bad=bad)


def tree_masks(parents, seq_lens, qsl, words):
    """(masks [T, words] as signed 32-bit, positions [T])."""
    masks, positions = [], []
    for s, L in enumerate(seq_lens):
        q0, n = qsl[s], qsl[s + 1] - qsl[s]
        paths = []
        for t in range(n):
            p = parents[q0 + t]
            path = (paths[p] if 0 <= p < t else 0) | 1 << t
            paths.append(path)
            row = [path >> (32 * w) & 0xFFFFFFFF for w in range(words)]
            masks.append([x - (1 << 32) if x >> 31 else x for x in row])
            positions.append(L - n + bin(path).count("1") - 1)
    return masks, positions


def attention(q, k, v, seen, scale):
    """q [n, 256], k and v [m, 256], seen bool [n, m] -> (out, sum of w |v|, log-sum-exp, sum of |q||k| scale), float64.
    Rows that see nothing: zeros, -inf."""
    x = np.where(seen, q @ k.T * scale, -np.inf)
    m = x.max(1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    w = np.exp(x - m)
    total = w.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(total))[:, 0]
    w = w / np.where(total > 0, total, 1.0)
    vz = np.where(seen.any(0)[:, None], v, 0.0)  # (what no row sees may be NaN)
    size = np.where(seen, np.abs(q) @ np.abs(k).T * abs(scale), 0.0).max(1, initial=0.0)
    return w @ vz, w @ np.abs(vz), lse, size


def tree_seen(masks, n, L):
    """bool [n, L] from a sequence's mask rows (signed 32-bit words)."""
    seen = np.zeros((n, L), dtype=bool)
    seen[:, :L - n] = True
    for t in range(n):
        for i in range(t + 1):
            seen[t, L - n + i] = masks[t][i // 32] >> (i % 32) & 1
    return seen
