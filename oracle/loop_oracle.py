"""Float64 / integer definitions of the operators around the layers (test infrastructure): rotary positions, the batch
plan and the verification of drafted tokens, token by token and request by request."""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------------------------------------
# rotary positions
# ------------------------------------------------------------------------------------------------
def frequencies(dim, theta=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0,
                low_turns=1.0, high_turns=4.0):
    """Radians a position of every pair."""
    if scaling == "base":
        theta = theta * factor ** (dim / (dim - 2))
    out = []
    for i in range(dim // 2):
        f = theta ** (-2.0 * i / dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            where = lambda turns: dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            low, high = max(math.floor(where(beta_fast)), 0), min(math.ceil(where(beta_slow)), dim - 1)
            r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = f * (r / factor + 1 - r)
        elif scaling == "bands":
            turns = original_len * f / (2 * math.pi)
            m = min(max((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0)
            f = f * ((1 - m) / factor + m)
        out.append(f)
    return np.array(out)


def angles(positions, freqs):
    """Angles in radians within (-pi, pi] from frequencies as 64-bit fractions of a turn (uint64)."""
    turns = (np.asarray(positions, np.int64).astype(np.uint64)[:, None] * np.asarray(freqs).view(np.uint64)[None]).view(np.int64)
    return turns.astype(np.float64) * 2.0 ** -64 * 2 * math.pi


def rope(x, positions, freqs, first=0, halves=False, inverse=False, scale=1.0):
    """x [T, heads, dim] float64, turned."""
    half = len(freqs)
    w = angles(positions, freqs)
    co, si = scale * np.cos(w), scale * np.sin(w) * (-1 if inverse else 1)
    y = x.astype(np.float64).copy()
    for i in range(half):
        a, b = (first + i, first + half + i) if halves else (first + 2 * i, first + 2 * i + 1)
        y[:, :, a] = x[:, :, a] * co[:, None, i] - x[:, :, b] * si[:, None, i]
        y[:, :, b] = x[:, :, b] * co[:, None, i] + x[:, :, a] * si[:, None, i]
    return y


# ------------------------------------------------------------------------------------------------
# batch plan
# ------------------------------------------------------------------------------------------------
class Cache:
    """One cache's numbers; plan() advances them in place."""

    def __init__(self, page, ratio, window, table, held, first, stack, count):
        self.page, self.ratio, self.window = page, ratio, window
        self.table, self.held, self.first = table.copy(), held.copy(), first.copy()
        self.stack, self.count = stack.copy(), int(count)

    def pages(self, rows):
        return -(-(rows // self.ratio) // self.page)


def plan(ctx, add, n_new, T, caches):
    """Returns a dict of ctx_out, q_start, kv_len, positions, seq, slots (one array a cache) and flagged."""
    B, flagged = len(ctx), False
    rows = [int(c) + int(a) for c, a in zip(ctx, add)]
    n = [int(x) for x in n_new]
    ok = []
    for b in range(B):
        good = rows[b] >= 0 and n[b] >= 0 and rows[b] + n[b] <= 2 ** 30
        for k in caches:
            if good:
                first, held, width = int(k.first[b]), int(k.held[b]), k.table.shape[1]
                good = 0 <= first <= held <= width and k.pages(rows[b] + n[b]) <= width
                if good and k.window and rows[b] + n[b] > 0:
                    good = max(0, rows[b] - k.window + 1) // k.page >= first
        ok.append(good)
        flagged |= not good
    held_before = [k.held.copy() for k in caches]
    for k in caches:
        size = len(k.stack)
        if not 0 <= k.count <= size:
            flagged, k.count = True, min(max(k.count, 0), size)
        for b in range(B):
            if not ok[b]:
                continue
            total, first, held = rows[b] + n[b], int(k.first[b]), int(k.held[b])
            if total == 0:
                back, lo, hi = range(first, held), 0, 0
            else:
                seen = max(0, rows[b] - k.window + 1) // k.page if k.window else 0
                lo = min(held, max(first, seen))
                hi = min(held, max(k.pages(total), lo))
                back = [*range(first, lo), *range(hi, held)]
            for j in back:
                if k.count < size:
                    k.stack[k.count] = k.table[b, j]
                    k.count += 1
                else:
                    flagged = True
            k.first[b], k.held[b] = lo, hi
    runs, tokens, wanted = [], 0, [0] * len(caches)
    for b in range(B):
        run = ok[b]
        if ok[b]:
            tokens += n[b]
            run = n[b] == 0 or tokens <= T
            for g, k in enumerate(caches):
                take = max(0, k.pages(rows[b] + n[b]) - int(held_before[g][b])) if n[b] else 0
                wanted[g] += take
                run = run and (take == 0 or wanted[g] <= k.count)
        runs.append(run)
    for g, k in enumerate(caches):
        for b in range(B):
            if not runs[b] or n[b] == 0:
                continue
            for j in range(int(held_before[g][b]), k.pages(rows[b] + n[b])):
                k.count -= 1
                k.table[b, j] = k.stack[k.count]
                flagged |= not 0 <= k.stack[k.count] < len(k.stack)
                k.held[b] = j + 1
    n = [x if r else 0 for x, r in zip(n, runs)]
    pos, seq = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    slots = [np.full(T, -1, np.int64) for _ in caches]
    t = 0
    q_start = [0]
    for b in range(B):
        for i in range(n[b]):
            pos[t], seq[t] = rows[b] + i, b
            for g, k in enumerate(caches):
                if (rows[b] + i + 1) % k.ratio == 0:
                    e = (rows[b] + i) // k.ratio
                    page = int(k.table[b, e // k.page])
                    if 0 <= page < len(k.stack):
                        slots[g][t] = page * k.page + e % k.page
            t += 1
        q_start.append(t)
    return {"ctx_out": np.array([rows[b] if ok[b] else int(ctx[b]) for b in range(B)], np.int32),
            "q_start": np.array(q_start, np.int32),
            "kv_len": np.array([rows[b] + n[b] if ok[b] else 0 for b in range(B)], np.int32),
            "positions": pos, "seq": seq, "slots": slots, "flagged": flagged}


# ------------------------------------------------------------------------------------------------
# verification of drafted tokens
# ------------------------------------------------------------------------------------------------
def law(row, probs, temperature, largest):
    """Probabilities and their logarithms of a row (float64 values of the stored type)."""
    x = np.asarray(row, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        if probs:
            p = np.where(np.isnan(x) | (x < 0), 0.0, np.minimum(x, largest))
            return p, np.log(p)
        x = np.where(np.isnan(x), -np.inf, np.minimum(x, largest))
        if x.max() == -np.inf:
            return np.zeros_like(x), np.full_like(x, -np.inf)
        z = (x - x.max()) / min(max(temperature, 1e-30), 1e30)
        z[x == -np.inf] = -np.inf
        total = np.exp(z).sum()
        return np.exp(z) / total, z - np.log(total)


def verify(target, tokens, q_start, width, draft=None, draft_row=None, temperature=None, u=None, noise=None,
           target_probs=False, draft_probs=False, largest=3.4028234663852886e38):
    """Returns out [B, width], count, logp, and margin [B]: how near (relatively) the nearest decision of a
    sequence was to the other one."""
    B, V = len(q_start) - 1, target.shape[1]
    out, logp = np.full((B, width), -1, np.int64), np.zeros((B, width))
    count, margin = np.zeros(B, np.int64), np.full(B, np.inf)
    drafted = int(q_start[0])  # tokens drafted for the sequences before, whose rows lie before this one's
    for b in range(B):
        t0, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        row0 = drafted
        drafted += max(n - 1, 0)
        temp = 1.0 if temperature is None else float(temperature[b])
        greedy = noise is None or not temp > 0
        for i in range(n):
            t = t0 + i
            p, lp = law(target[t], target_probs, 1.0 if greedy else temp, largest)
            first = int(np.argmax(np.where(np.isnan(target[t]), -np.inf, np.minimum(target[t], largest)))) if p.max() > 0 else -1
            left, x = p, int(tokens[t + 1]) if i + 1 < n else -1
            if i + 1 < n:
                known, q, lq = True, np.zeros(V), None
                if draft is not None and not greedy:
                    d = int(draft_row[t + 1]) if draft_row is not None else row0 + i
                    known = 0 <= d < len(draft)
                    if known:
                        q, lq = law(draft[d], draft_probs, temp, largest)
                        left = np.maximum(p - q, 0)
                elif not greedy:
                    left = p.copy()
                    if 0 <= x < V:
                        left[x] = 0
                ok = False
                if 0 <= x < V:
                    if greedy:
                        ok = x == first
                    elif known:
                        # u q < p by logarithms: both sides may be too small for a float64
                        with np.errstate(divide="ignore", invalid="ignore"):
                            limit = np.log(np.float64(u[t + 1])) + (0.0 if draft is None else lq[x])
                            ok = bool(lp[x] > -np.inf and limit < lp[x])
                            if lp[x] > -np.inf and limit > -np.inf:
                                margin[b] = min(margin[b], abs(limit - lp[x]))
                if ok:
                    out[b, i], logp[b, i] = x, lp[x]
                    continue
            count[b] = i
            if greedy:
                y = first
            else:
                if left.max() <= 0:
                    left = p
                key = left / noise[b].astype(np.float64)
                y = int(np.argmax(key)) if key.max() > 0 else -1
                if y >= 0 and V > 1:
                    second = np.partition(key, V - 2)[V - 2]
                    # (a difference p - q is as near to another as its terms are large beside it)
                    margin[b] = min(margin[b], (key[y] - second) / key[y] * min(1.0, left[y] / p[y]))
            if y >= 0:
                out[b, i], logp[b, i], count[b] = y, lp[y], i + 1
            break
    return out, count, logp, margin
