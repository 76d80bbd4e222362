"""Seeded small inputs of the grouped-query operators, shared by their CPU and GPU tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import dsv4_oracle as O

E4M3_NAN, BF16_NAN = 0x7F, 0x7FC0


class Batch:
    """Paged caches filled for sequences of kv[b] rows whose last n[b] are new, every row that belongs to no
    sequence NaN.  Arrays are numpy (bf16 as uint16 bits, e4m3 as uint8 codes)."""

    def __init__(self, n, kv, H, Hkv, D, page, cache, seed=0, qscale=1.0, pad=0, spare_pages=2):
        g = np.random.default_rng(seed)
        self.n, self.kv = np.asarray(n, np.int32), np.asarray(kv, np.int32)
        self.H, self.Hkv, self.D, self.page, self.cache = H, Hkv, D, page, cache
        B = len(n)
        self.q_start = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.T = int(self.q_start[-1]) + pad
        used = -(-self.kv // page)
        width = max(1, int(used.max(initial=0)))
        pages = int(used.sum()) + spare_pages
        order = g.permutation(pages)
        self.table = np.full((B, width), 2 ** 30, np.int32)   # entries behind a sequence's rows are never read
        at = 0
        for b in range(B):
            self.table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
        bf = lambda *s: O.bf16_encode(g.standard_normal(s))  # noqa: E731
        self.q = O.bf16_encode(g.standard_normal((self.T, H, D)) * qscale)
        self.k_new, self.v_new = bf(self.T, Hkv, D), bf(self.T, Hkv, D)
        shape = (pages, Hkv, page, D)
        self.caches, self.exps = [], None if cache == "bf16" else []
        for _ in range(2):
            if cache == "bf16":
                c = np.full(shape, BF16_NAN, np.uint16)
                fresh = bf(*shape)
            else:
                c = np.full(shape, E4M3_NAN, np.uint8)
                fresh = O.e4m3_encode(np.clip(g.standard_normal(shape) * 100, -448, 448))
                e = g.integers(117, 123, (pages, Hkv)).astype(np.uint8)
                free = np.ones(pages, bool)
                free[order[:at]] = False
                e[free] = 255
                self.exps.append(e)
            for b in range(B):
                for i in range(used[b]):
                    rows = min(page, int(self.kv[b]) - i * page)
                    c[self.table[b, i], :, :rows] = fresh[self.table[b, i], :, :rows]
            self.caches.append(c)
        self.max_q, self.max_kv = max(1, int(self.n.max(initial=0))), int(self.kv.max(initial=0))

    def q64(self):
        return O.bf16_decode(self.q).astype(np.float64)


def dev(a, device="cuda"):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(a).to(device)


def host(t):
    if t.dtype == torch.bfloat16:
        return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


def strided(t, layout):
    """The cache tensor's values behind another memory order: 'hnd' as it is, 'nhd' with the rows of a page
    outside its heads, 'wide' with rows, heads and pages apart from one another."""
    if layout == "hnd":
        return t
    if layout == "nhd":
        return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    pages, heads, rows, dim = t.shape
    big = torch.zeros((pages, heads + 1, rows + 1, 2 * dim), dtype=t.dtype, device=t.device)
    view = big[:, :heads, :rows, dim:]
    view.copy_(t)
    return view


def bounds(mag, size, out, lse, bf16_out, p_bits=8):
    """Largest errors that the kernels' roundings add up to.  A logit: products exact, at most 128 fp32
    additions in any order or with truncated alignment (2^-16 of sum |q k|), then a handful of fp32 roundings
    of z and of the exponent's argument (2^-20 (1 + |z|)).  Its weight moves by as much, relatively, and the
    normalised weight by twice that.  A weight rounded to bf16 or fp16 before the product with V moves by half
    a step (2^-8, the larger), the sums over V as the logits' do (2^-13 of sum w |v|: one tile's sum at a time,
    then rescaled fp32 additions over at most 2^10 tiles).  The output's own rounding: 2^-8 bf16."""
    dz = 2.0 ** -16 * size + 2.0 ** -20 * (1 + size)
    tol = mag * (2 * np.expm1(dz)[..., None] + 2.0 ** -p_bits + 2.0 ** -13) + 1e-30
    if bf16_out:
        tol = tol + 2.0 ** -8 * (np.abs(out) + tol)
    return tol, dz + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
