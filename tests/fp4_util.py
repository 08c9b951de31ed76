"""4-bit caches for the tests: built from the oracle's format, compared with its values."""
from __future__ import annotations

import dataclasses
from typing import List, Tuple

import numpy as np
import torch

import oracle
from oracle import fp4

D = 256


@dataclasses.dataclass
class Fp4Case:
    seqs: List[Tuple[int, int]]  # (q_len, L)
    hq: int
    hkv: int
    page: int
    q: torch.Tensor
    k: torch.Tensor              # uint8 [NB, Hkv, P, 144]
    v: torch.Tensor
    table: torch.Tensor
    lens: torch.Tensor
    qsl: torch.Tensor
    kd: float
    vd: float
    scale: float = 1.0 / 16.0

    @property
    def T(self):
        return int(self.qsl[-1])


def make(seqs, hq, hkv, page, seed=0, device="cuda", kd=0.01, vd=0.02, spare=3, poison=True, size=1.0) -> Fp4Case:
    """A batch on caches of quantised N(0, size) values; slots that no sequence holds are 0xFF
    (NaN scales), block-table entries past a sequence's pages -1."""
    rng = np.random.default_rng(1000 + seed)
    n_pages = [-(-L // page) for _, L in seqs]
    NB = max(1, sum(n_pages) + spare)
    W = max([1] + n_pages) + 1
    perm = rng.permutation(NB)
    bt = np.full((len(seqs), W), -1, dtype=np.int32)
    held = np.zeros((NB, page), dtype=bool)
    at = 0
    for s, (_, L) in enumerate(seqs):
        mine = perm[at:at + n_pages[s]]
        bt[s, :len(mine)] = mine
        for i, p in enumerate(mine):
            held[p, :min(page, L - i * page)] = True
        at += n_pages[s]
    caches = []
    for is_v, descale in ((False, kd), (True, vd)):
        x = rng.standard_normal((NB, page, hkv, D), dtype=np.float32) * np.float32(size)
        codes, s8 = fp4.quantise(x, descale)
        if poison:
            codes[~held], s8[~held] = 15, 255
        caches.append(torch.from_numpy(fp4.pack(codes, s8, is_v)))
    T = sum(q for q, _ in seqs)
    q = torch.from_numpy(rng.standard_normal((T, hq, D), dtype=np.float32)).bfloat16()
    qsl = torch.tensor([0] + list(np.cumsum([q_ for q_, _ in seqs])), dtype=torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    return Fp4Case(list(seqs), hq, hkv, page, q.to(device), caches[0].to(device), caches[1].to(device),
                   torch.from_numpy(bt).to(device), lens.to(device), qsl.to(device), kd, vd)


def dequantised(case: Fp4Case):
    """code * scale of both caches as bf16 [NB, P, Hkv, 256] (exact: 6 significant bits)."""
    out = []
    for t, is_v in ((case.k, False), (case.v, True)):
        x = fp4.values(*fp4.unpack(t.cpu().numpy(), is_v))
        b = torch.from_numpy(x).to(torch.bfloat16)
        same = (b.double() == torch.from_numpy(x)) | torch.from_numpy(np.isnan(x))
        assert bool(same.all())
        out.append(b)
    return out


def reference(case: Fp4Case, rows=None):
    """The 64-bit attention of the case: out [T, Hq, 256] (or the listed rows)."""
    k, v = dequantised(case)
    return oracle.attention(case.q.cpu(), k, v, case.table.cpu(), case.lens.cpu(), case.qsl.cpu(), q_dtype="bf16",
                            kv_dtype="bf16", q_descale=1.0, k_descale=float(np.float32(case.kd)),
                            v_descale=float(np.float32(case.vd)), softmax_scale=case.scale, rows=rows)


def v_max(case: Fp4Case) -> float:
    """The largest |V| that the batch holds."""
    x = np.abs(fp4.values(*fp4.unpack(case.v.cpu().numpy(), True)))
    return float(np.nanmax(x)) * case.vd


def check(case: Fp4Case, got: torch.Tensor, what: str, rows=None):
    """Each output within its own arithmetic's bound of the 64-bit value:
      the output's bf16 rounding           2^-8 |o|
      P rounded to 11 bits before P.V      2^-11 sum p |v| / sum p <= 2^-11 max |v|
      (and in the row sums, which use the rounded P or differ by as much)      2^-11 |o|
      a split piece's f16 partial          2^-11 max |v|
      fp32 sums and the exponential, over <= 2^16 keys: below 2^-12 max |v| together
    """
    ref = reference(case, rows)
    g = got.detach().float().cpu().numpy().astype(np.float64).reshape(-1, D)
    if rows is not None:
        g = g[np.asarray(rows)]
    g = g.reshape(ref.shape)
    assert np.isfinite(g).all(), f"{what}: {(~np.isfinite(g)).sum()} values are not finite"
    bound = (2.0 ** -8 + 2.0 ** -11) * np.abs(ref) + 2.0 ** -9.5 * v_max(case)
    off = np.abs(g - ref) - bound
    assert (off <= 0).all(), f"{what}: {(off > 0).sum()} values off, worst by {off.max():.3g} over its bound"
    norm = float(np.linalg.norm(ref)) or 1.0
    rel = float(np.linalg.norm(g - ref)) / norm
    assert rel <= 5e-3, f"{what}: rel-L2 {rel:.3g}"
    return rel
