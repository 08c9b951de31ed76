"""Oracle of the 4-bit paged cache (TEST INFRASTRUCTURE ONLY).

Only ``tests/`` and ``__graft_entry__.smoke()`` may import this module; the CUDA library never
does, and this module never imports it.

The format, from its definition: 256 values of a (token, kv head) are 128 bytes of e2m1 codes
(1 sign, 2 exponent bits with bias 1, 1 fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; byte i holds
d = 2i in its low nibble and d = 2i + 1 in its high one) and 16 e4m3 scales, one per 16 values;
value = code * scale * descale. Caches are uint8 [NB, Hkv, P, 144]: K pages hold token after
token [128 codes][16 scales], V pages blocks of 16 tokens, code byte i of token j at
i * 16 + j and the scale of group g at 2048 + g * 16 + j.

A write takes, per group of 16 values in float32: y = x * inv (inv = 1 / descale rounded first),
scale = e4m3(max |y| * float32(1/6)) at most 448, code = e2m1(y * r) with r = 1 / scale rounded
(0 for a zero scale), both to nearest even, codes at most 6. A NaN makes the group's scale NaN.

Parity status: pinned (tests/test_fp4_oracle.py: every code and scale decoded, ties, saturation,
agreement with torch.float8_e4m3fn, the packing against a loop over single values).
"""
from __future__ import annotations

import numpy as np

from .cache_write import e4m3_encode

ROW = 144
BLOCK = 16
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def code_value(c: np.ndarray) -> np.ndarray:
    """e2m1 codes 0..15 -> float64."""
    c = np.asarray(c).astype(np.int64)
    return np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]


def scale_value(b: np.ndarray) -> np.ndarray:
    """e4m3 bytes -> float64 (0x7F and 0xFF are NaN)."""
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * np.exp2(e - 7.0))
    return np.where((b & 127) == 127, np.nan, np.where(b & 128, -x, x))


def encode(y: np.ndarray) -> np.ndarray:
    """Values -> e2m1 codes: the nearest level, a tie to the even code, at most 6 in size."""
    y = np.asarray(y, dtype=np.float32)
    a = np.where(np.isnan(y), 7.0, np.abs(y.astype(np.float64)))
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    n = np.zeros(a.shape, dtype=np.uint8)
    for i, m in enumerate(mid):  # between codes i and i + 1: a tie goes to the even one
        n += (a > m) if i % 2 == 0 else (a >= m)
    return np.where(np.signbit(y) & ~np.isnan(y), n + 8, n).astype(np.uint8)


def quantise(x: np.ndarray, descale: float):
    """[..., 256] float32 -> (codes [..., 256] 0..15, scale bytes [..., 16])."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        y = (x * (np.float32(1.0) / np.float32(descale))).reshape(*x.shape[:-1], 16, 16)
        top = np.max(np.abs(y), axis=-1)  # NaN if any is
        s8 = e4m3_encode(top * np.float32(1.0 / 6.0))
        s = scale_value(s8).astype(np.float32)
        r = np.where(s == 0, np.float32(0), np.float32(1) / s).astype(np.float32)
        codes = encode(y * r[..., None])
    return codes.reshape(x.shape), s8


def values(codes: np.ndarray, s8: np.ndarray) -> np.ndarray:
    """codes [..., 256], scale bytes [..., 16] -> float64 code * scale."""
    return code_value(codes) * np.repeat(scale_value(s8), 16, axis=-1)


def _token(page: np.ndarray, slot: int, is_v: bool):
    """Index arrays of a token's code bytes and scale bytes inside a page's flat bytes."""
    if not is_v:
        return slot * ROW + np.arange(128), slot * ROW + 128 + np.arange(16)
    base, j = slot // BLOCK * BLOCK * ROW, slot % BLOCK
    return base + np.arange(128) * BLOCK + j, base + 2048 + np.arange(16) * BLOCK + j


def put(cache: np.ndarray, page: int, head: int, slot: int, is_v: bool, codes: np.ndarray, s8: np.ndarray) -> None:
    """Store one token's codes [256] and scales [16]."""
    flat = cache[page, head].reshape(-1)
    ci, si = _token(flat, slot, is_v)
    flat[ci] = codes[0::2] | (codes[1::2] << 4)
    flat[si] = s8


def unpack(cache: np.ndarray, is_v: bool):
    """A whole cache -> codes [NB, P, Hkv, 256], scale bytes [NB, P, Hkv, 16]."""
    NB, H, P, _ = cache.shape
    if is_v:
        b = cache.reshape(NB, H, P // BLOCK, BLOCK * ROW)
        cb = b[..., :2048].reshape(NB, H, P // BLOCK, 128, BLOCK).swapaxes(-1, -2).reshape(NB, H, P, 128)
        s8 = b[..., 2048:].reshape(NB, H, P // BLOCK, 16, BLOCK).swapaxes(-1, -2).reshape(NB, H, P, 16)
    else:
        cb, s8 = cache[..., :128], cache[..., 128:]
    codes = np.stack([cb & 15, cb >> 4], axis=-1).reshape(NB, H, P, 256)
    return codes.swapaxes(1, 2), s8.swapaxes(1, 2)


def pack(codes: np.ndarray, s8: np.ndarray, is_v: bool) -> np.ndarray:
    """The inverse of unpack."""
    codes, s8 = codes.swapaxes(1, 2), s8.swapaxes(1, 2)
    NB, H, P, _ = codes.shape
    cb = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    if not is_v:
        return np.ascontiguousarray(np.concatenate([cb, s8], axis=-1))
    cb = cb.reshape(NB, H, P // BLOCK, BLOCK, 128).swapaxes(-1, -2).reshape(NB, H, P // BLOCK, 2048)
    s8 = s8.reshape(NB, H, P // BLOCK, BLOCK, 16).swapaxes(-1, -2).reshape(NB, H, P // BLOCK, 256)
    return np.ascontiguousarray(np.concatenate([cb, s8], axis=-1)).reshape(NB, H, P, ROW)


def write(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale, v_descale):
    """Copies of the caches with the new tokens [T, Hkv, 256] (float32 of the bf16 inputs) written."""
    kc, vc = k_cache.copy(), v_cache.copy()
    P = kc.shape[2]
    kq, vq = quantise(k_new, k_descale), quantise(v_new, v_descale)
    for s in range(len(seq_lens)):
        q0, q1 = int(query_start_loc[s]), int(query_start_loc[s + 1])
        for t in range(q0, q1):
            pos = int(seq_lens[s]) - (q1 - t)
            page, slot = int(block_table[s, pos // P]), pos % P
            for h in range(kc.shape[1]):
                put(kc, page, h, slot, False, kq[0][t, h], kq[1][t, h])
                put(vc, page, h, slot, True, vq[0][t, h], vq[1][t, h])
    return kc, vc


def read(k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale, v_descale):
    """float64 K and V [T, Hkv, 256] of the last tokens of each sequence."""
    P, H = k_cache.shape[2], k_cache.shape[1]
    T = int(query_start_loc[-1])
    out = []
    for cache, is_v, descale in ((k_cache, False, k_descale), (v_cache, True, v_descale)):
        x = values(*unpack(cache, is_v)) * float(np.float32(descale))
        o = np.zeros((T, H, 256))
        for s in range(len(seq_lens)):
            q0, q1 = int(query_start_loc[s]), int(query_start_loc[s + 1])
            for t in range(q0, q1):
                pos = int(seq_lens[s]) - (q1 - t)
                o[t] = x[int(block_table[s, pos // P]), pos % P]
        out.append(o)
    return out[0], out[1]
