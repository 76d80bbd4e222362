"""Plain CPU oracle of the grouped-query operators (test infrastructure only): the append of rotated
keys and values to paged per-head caches and the attention over them, sequence by sequence in numpy
float64 on exactly decoded values.  The rotation is the definition's own fp32 arithmetic (every product
and sum rounded), so stored codes and exponents are exact.
"""
from __future__ import annotations

import numpy as np

from .dsv4_oracle import bf16_decode, bf16_encode, e4m3_decode, e4m3_encode, ue8m0_exponent


def rotate(x, pos: int, cos_sin, first: int, halves: bool) -> np.ndarray:
    """fp32 rows x [..., dim] at one position; cos_sin [max_pos, rope_dim] or None."""
    x = np.asarray(x, np.float32).copy()
    if cos_sin is None:
        return x
    half = cos_sin.shape[1] // 2
    co, si = cos_sin[pos, :half], cos_sin[pos, half:]
    i = np.arange(half)
    ia, ib = (first + i, first + half + i) if halves else (first + 2 * i, first + 2 * i + 1)
    a, b = x[..., ia], x[..., ib]
    x[..., ia] = a * co - b * si
    x[..., ib] = b * co + a * si
    return x


def page_exponent(amax: float) -> int:
    return -127 if amax == 0 else max(-127, ue8m0_exponent(amax))


def append(k_new, v_new, caches, exps, table, q_start, kv_len, cos_sin=None, first=0, halves=False):
    """Stores fp32 rows k_new, v_new [T, heads, dim] into caches = [k, v] ([pages, heads, page_size, dim] bf16
    bits, or e4m3 codes with exps = [k, v] bytes), in place."""
    page_size = caches[0].shape[2]
    for b in range(len(kv_len)):
        n = int(q_start[b + 1] - q_start[b])
        p0 = int(kv_len[b]) - n
        for c, new in enumerate((k_new, v_new)):
            rows = [rotate(new[q_start[b] + i], p0 + i, cos_sin, first, halves) if c == 0 else
                    np.asarray(new[q_start[b] + i], np.float32) for i in range(n)]
            for lp in range(p0 // page_size, (p0 + n - 1) // page_size + 1 if n else 0):
                page = int(table[b, lp])
                lo, hi = max(lp * page_size, p0), min((lp + 1) * page_size, p0 + n)
                for h in range(new.shape[1]):
                    part = np.stack([rows[j - p0][h] for j in range(lo, hi)])
                    r0 = lo - lp * page_size
                    if exps is None:
                        caches[c][page, h, r0:r0 + len(part)] = bf16_encode(part)
                        continue
                    e = page_exponent(float(np.abs(part).max()))
                    if r0 > 0:
                        old = int(exps[c][page, h]) - 127
                        e = max(e, old)
                        if e > old:
                            held = e4m3_decode(caches[c][page, h, :r0])
                            caches[c][page, h, :r0] = e4m3_encode(held * 2.0 ** (old - e))
                    exps[c][page, h] = e + 127
                    caches[c][page, h, r0:r0 + len(part)] = e4m3_encode(part.astype(np.float64) * 2.0 ** -e)


def rows_of(cache, exp, table_b, h: int, kv: int) -> np.ndarray:
    """The first kv rows of kv head h of a sequence, float64."""
    page_size = cache.shape[2]
    out = np.empty((kv, cache.shape[3]))
    for j0 in range(0, kv, page_size):
        page, n = int(table_b[j0 // page_size]), min(page_size, kv - j0)
        x = bf16_decode(cache[page, h, :n]) if exp is None else \
            e4m3_decode(cache[page, h, :n]) * 2.0 ** (int(exp[page, h]) - 127)
        out[j0:j0 + n] = x
    return out


def attention(q, caches, exps, table, q_start, kv_len, scale, causal=True, prefix_len=None, kv_start=None, window=0,
              softcap=0.0, slopes=None, sink=None):
    """out [T, H, dim], lse [T, H] in float64, and per (token, head) two magnitudes that error bounds are made
    of: sum_j w_j |v_j| ([T, H, dim]) and max_j scale * sum_i |q_i k_ji|, the largest |z| included ([T, H])."""
    T, H, dim = q.shape
    out, lse = np.zeros((T, H, dim)), np.full((T, H), -np.inf)
    mag, size = np.zeros((T, H, dim)), np.zeros((T, H))
    heads = caches[0].shape[1]
    group = H // heads
    for b in range(len(kv_len)):
        t0, t1, kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        j = np.arange(kv)
        for hk in range(heads):
            k = rows_of(caches[0], None if exps is None else exps[0], table[b], hk, kv)
            v = rows_of(caches[1], None if exps is None else exps[1], table[b], hk, kv)
            for t in range(t0, t1):
                p = kv - (t1 - t0) + t - t0
                see = np.ones(kv, bool)
                if causal:
                    see = j <= p
                    if prefix_len is not None:
                        see |= j < prefix_len[b]
                if window:
                    see &= j > p - window
                if kv_start is not None:
                    see &= j >= kv_start[t]
                for h in range(hk * group, hk * group + group):
                    s = -np.inf if sink is None else float(sink[h])
                    z = k[see] @ q[t, h] * scale
                    big = np.abs(k[see]) @ np.abs(q[t, h]) * abs(scale)
                    if softcap:
                        z = softcap * np.tanh(z / softcap)
                    if slopes is not None:
                        z = z - float(slopes[h]) * np.abs(p - j[see])
                    m = max(s, z.max() if z.size else -np.inf)
                    if m == -np.inf:
                        continue
                    w = np.exp(z - m)
                    total = w.sum() + np.exp(s - m)
                    out[t, h] = w @ v[see] / total
                    mag[t, h] = w @ np.abs(v[see]) / total
                    lse[t, h] = m + np.log(total)
                    size[t, h] = max(big.max(), np.abs(z).max()) if z.size else 0.0
    return out, lse, mag, size
