"""Measured cases of the grouped-query operators: appending rotated keys and values to a paged cache
(bfloat16, or e4m3 codes with one power-of-two scale for each page and head), and attention of one or
many new tokens a sequence over that cache.

`run` computes an operator in plain float32 torch operations, or, with `own` true, through the
package's calls.  `exact` is the same definition in float64, written sequence by sequence.

Layout of a case: sequence b holds `kv_len[b]` rows after the call, the last `n[b]` of them new; new
token i of b (flat index q_start[b] + i) is at position kv_len[b] - n[b] + i.  A token at position p
sees row j when  j < kv_len, (not causal or j <= p or j < prefix_len[b]), (no window or j > p - window)
and j >= kv_start[token] (the start of its document).
"""
import math

import numpy as np
import torch

own = False

_BASE = {"H": 64, "Hkv": 8, "D": 128, "page": 64, "cache": "fp8", "spread": 0.0, "window": 0, "softcap": 0.0,
         "alibi": False, "sink": False, "docs": 0, "prefix": 0, "qscale": 1.0, "rope": 128, "halves": False,
         "ctx": 0, "n_spread": 0.0}


def _case(op, **kw):
    c = dict(_BASE)
    c["op"] = op
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of 32 running sequences: queries rotated, one key and value row a sequence stored
        _case("append", name="append_step_32", B=32, n=1, ctx=4095, spread=0.9),
        # four ragged prompts stored at once behind earlier rows (chunked prefill), pages entered mid-way
        _case("append", name="append_prompts_fp8", B=4, n=4096, n_spread=0.7, ctx=1000, spread=0.5),
        # halves-style rotation of part of a 64-wide head, bf16 cache in small pages, five queries a key head
        _case("append", name="append_prompts_bf16", B=9, n=701, n_spread=0.9, ctx=77, spread=0.9, H=20, Hkv=4, D=64,
              page=16, cache="bf16", rope=32, halves=True),
        # the smallest serving call: one sequence, one token, a short context
        _case("attend", name="decode_1x777_fp8", B=1, n=1, ctx=776),
        # a serving batch of mixed lengths
        _case("attend", name="decode_32x8k_fp8", B=32, n=1, ctx=8191, spread=0.9),
        # four tokens a sequence to verify (draft decoding), window and capped scores, bf16 cache
        _case("attend", name="decode_mtp4_cap_bf16", B=48, n=4, ctx=4000, spread=0.5, H=32, Hkv=4, cache="bf16",
              window=1024, softcap=30.0, qscale=4.0, sink=True),
        # many short sequences of one shared key head with distance bias, 64-wide heads, small pages
        _case("attend", name="decode_200_alibi_mqa", B=200, n=1, ctx=1500, spread=0.95, H=16, Hkv=1, D=64, page=16,
              alibi=True),
        # few very long contexts
        _case("attend", name="decode_4x128k_fp8", B=4, n=1, ctx=131070, spread=0.1),
        # short odd prompts with a bidirectional prefix, packed documents, a key head for each query head
        _case("attend", name="prefill_3x129_docs", B=3, n=129, n_spread=0.8, ctx=30, H=12, Hkv=12, D=64, page=32,
              cache="bf16", docs=50, prefix=17),
        # a chunk of two long prompts against their earlier rows
        _case("attend", name="prefill_chunk_512_of_32k", B=2, n=512, n_spread=0.2, ctx=32400, spread=0.3),
        # packed documents with capped scores, bf16 cache
        _case("attend", name="prefill_cap_docs_bf16", B=2, n=4096, n_spread=0.5, ctx=0, H=32, cache="bf16", docs=1100,
              softcap=50.0, qscale=4.0),
        # one long prompt, causal
        _case("attend", name="prefill_8k_fp8", B=1, n=8192, ctx=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "prefill", "prefill"])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    D = rng.choice([64, 128, 128])
    c = {"H": Hkv * group, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 64, 128]),
         "cache": rng.choice(["fp8", "fp8", "bf16"]), "spread": rng.choice([0.0, 0.5, 0.9])}
    if kind == "append":
        n = rng.choice([1, rng.randint(2, 5), _log(rng, 6, 4096)])
        c["rope"] = rng.choice([D, D // 2, 0])
        c["halves"] = rng.random() < 0.5
        return _case("append", B=max(1, min(64, _log(rng, 1, 16384) // n)), n=n, n_spread=rng.choice([0.0, 0.8]),
                     ctx=_log(rng, 1, 2048) - 1, **c)
    c["window"] = rng.choice([0, 0, _log(rng, 100, 5000)])
    c["softcap"] = rng.choice([0.0, 0.0, 20.0])
    c["qscale"] = 4.0 if c["softcap"] else 1.0
    c["alibi"] = rng.random() < 0.25
    c["sink"] = rng.random() < 0.25
    if kind == "decode":
        ctx = _log(rng, 1, 100000) - 1
        most = max(1, 400000 * 8 // (Hkv * (ctx + 1)))
        return _case("attend", B=min(_log(rng, 1, 256), most), n=rng.choice([1, 1, 2, 4]), ctx=ctx, **c)
    n = _log(rng, 5, 6000)
    ctx = rng.choice([0, 0, _log(rng, 1, 8000)])
    most = max(1, int(8192 * 8192 * 32 // (c["H"] * n * (ctx + n))))
    while most == 1 and c["H"] * n * (ctx + n) > 8192 * 8192 * 32:
        n, ctx = max(1, n // 2), ctx // 2
    return _case("attend", B=min(_log(rng, 1, 12), most), n=n, n_spread=rng.choice([0.0, 0.8]), ctx=ctx,
                 docs=rng.choice([0, 0, _log(rng, 20, 2000)]), prefix=rng.choice([0, 0, _log(rng, 2, 500)]), **c)


def _lens(B, top, spread):
    """Ragged lengths: the first is `top`, the others lie between top * (1 - spread) and top."""
    return np.floor(top * (1.0 - spread * np.mod(np.arange(B) * 0.6180339887, 1.0))).astype(np.int64)


def _layout(c):
    B = c["B"]
    n = np.maximum(1, _lens(B, c["n"], c["n_spread"]))
    ctx = _lens(B, c["ctx"], c["spread"])
    q_start = np.concatenate([[0], np.cumsum(n)])
    seq = np.repeat(np.arange(B), n)
    pos = np.arange(q_start[-1]) - q_start[seq] + ctx[seq]
    start = pos // c["docs"] * c["docs"] if c["docs"] else np.zeros_like(pos)
    prefix = np.minimum(c["prefix"], ctx + n) if c["prefix"] else np.zeros(B, np.int64)
    return {"n": n, "kv": ctx + n, "q_start": q_start, "seq": seq, "pos": pos, "start": start, "prefix": prefix}


def _seen(c, L):
    """First row and number of rows that each token sees (the rows a token sees are contiguous)."""
    lo = L["start"]
    if c["window"]:
        lo = np.maximum(lo, L["pos"] - c["window"] + 1)
    hi = np.maximum(L["pos"] + 1, L["prefix"][L["seq"]])
    return lo, np.maximum(0, np.minimum(hi, L["kv"][L["seq"]]) - lo)


def work(case):
    c, L = case, _layout(case)
    T, H, Hkv, D = len(L["pos"]), c["H"], c["Hkv"], c["D"]
    size = 1 if c["cache"] == "fp8" else 2
    if c["op"] == "append":
        return {"bytes": T * D * (4 * H + 2 * Hkv * (2 + size)), "flops": 3 * T * D * (H + Hkv)}
    lo, count = _seen(c, L)
    first, last = np.full(c["B"], 1 << 60), np.zeros(c["B"], np.int64)
    np.minimum.at(first, L["seq"], lo)
    np.maximum.at(last, L["seq"], lo + count)
    rows = int(np.maximum(0, last - first).sum())
    return {"bytes": 4 * T * H * D + 4 * T * H + rows * Hkv * 2 * D * size, "flops": 4 * D * H * int(count.sum())}


def prepare(case, seed):
    c, L = case, _layout(case)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, H, Hkv, D, P = c["B"], c["H"], c["Hkv"], c["D"], c["page"]
    T = len(L["pos"])
    width = int(-(-L["kv"].max() // P))
    used = -(-L["kv"] // P)
    pages = int(used.sum()) + 3
    order = torch.randperm(pages, generator=g, device=dev)
    table = torch.zeros((B, width), dtype=torch.int64, device=dev)
    held = torch.from_numpy(np.arange(width)[None, :] < used[:, None]).to(dev)
    table[held] = order[: int(used.sum())]
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev).to(torch.int32)  # noqa: E731
    s = {"case": c, "table": table.to(torch.int32), "q_start": ints(L["q_start"]), "kv_len": ints(L["kv"]),
         "max_q": int(L["n"].max()), "max_kv": int(L["kv"].max())}
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    # queries, keys and values come out of one projection: rows of a fused [T, H + 2 Hkv, D] buffer
    qkv = normal(T, H + 2 * Hkv, D).to(torch.bfloat16)
    if c["op"] == "attend" and c["qscale"] != 1.0:
        qkv[:, :H] *= c["qscale"]
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    for name in ("k", "v"):
        if c["cache"] == "fp8":
            codes = torch.empty((pages, Hkv, P, D), dtype=torch.float8_e4m3fn, device=dev)
            for part in codes.view(torch.uint8).split(max(1, (1 << 27) // (Hkv * P * D))):
                part.copy_((normal(*part.shape) * 96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            s[name + "_cache"] = codes
            s[name + "_scale"] = torch.randint(118, 122, (pages, Hkv), generator=g, device=dev, dtype=torch.uint8)
        else:
            s[name + "_cache"] = normal(pages, Hkv, P, D).to(torch.bfloat16)
            s[name + "_scale"] = None
    if c["op"] == "append":
        half = c["rope"] // 2
        s["cos_sin"] = None
        if half:
            freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
            angle = torch.arange(s["max_kv"], dtype=torch.float64, device=dev)[:, None] * freq
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    else:
        s["scale"] = D ** -0.5
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev) / H) if c["alibi"] else None
        s["sink"] = normal(H) if c["sink"] else None
        s["prefix_len"] = ints(L["prefix"]) if c["prefix"] else None
        s["kv_start"] = ints(L["start"]) if c["docs"] else None
        s["out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device=dev)
    return s


def run(s):
    append = s["case"]["op"] == "append"
    if own:
        return _own_append(s) if append else _own_attend(s)
    return _plain_append(s) if append else _plain_attend(s)


# ------------------------------------------------------------------------------------------------
# the package's calls.  As in a decode loop over fixed buffers, a call's parameters are filled in on
# the first pass over a state and kept beside its buffers.
# ------------------------------------------------------------------------------------------------
def _own_append(s):
    import deepseek_v4_hybrid_gb300 as M
    if "plan" not in s:
        c = s["case"]
        s["plan"] = M.gqa_append_params(
            s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"], s["max_q"],
            k_scale=s["k_scale"], v_scale=s["v_scale"], cos_sin=s["cos_sin"], rope_first=c["D"] - c["rope"],
            rope_halves=c["halves"], q=s["q"], q_out=s["q_out"])
    M.dsv4_gqa_append(s["plan"])
    return _append_outputs(s)


def _own_attend(s):
    import deepseek_v4_hybrid_gb300 as M
    if "plan" not in s:
        c = s["case"]
        p = M.gqa_attention_params(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"], s["max_q"], s["max_kv"],
            s["scale"], s["out"], lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"], window=c["window"],
            softcap=c["softcap"], slopes=s["slopes"], sink=s["sink"], prefix_len=s["prefix_len"],
            kv_start=s["kv_start"])
        s["workspace"] = torch.empty(M.dsv4_gqa_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        M.gqa_set_workspace(p, s["workspace"])
        s["plan"] = p
    M.dsv4_gqa_attention(s["plan"])
    return {"out": s["out"], "lse": s["lse"]}


def _append_outputs(s):
    """The rotated queries and both caches: e4m3 codes as the numbers they stand for in units of their
    page's and head's scale, and beside them the scales' exponents (whole numbers)."""
    r = {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if s["k_scale"] is not None:
        r.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return r


# ------------------------------------------------------------------------------------------------
# plain form, float32
# ------------------------------------------------------------------------------------------------
def _rotate(x, cs, halves):
    """The last 2 * half dims of x [T, heads, D] turned by cos | sin rows cs [T, 2 * half]."""
    x = x.float()
    if cs is None:
        return x
    half = cs.shape[1] // 2
    first = x.shape[-1] - 2 * half
    a, b = (x[..., first:first + half], x[..., first + half:]) if halves else (x[..., first::2], x[..., first + 1::2])
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    y = x.clone()
    if halves:
        y[..., first:first + half], y[..., first + half:] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., first::2], y[..., first + 1::2] = a * cos - b * sin, b * cos + a * sin
    return y


def _exponent(amax):
    """Smallest e >= -127 with 448 * 2^e >= amax (-127 for an all-zero block): 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), -127).clamp(min=-127).to(torch.int32)


def _token_places(s):
    """Sequence, cache position, page and row in the page of every new token."""
    q_start, kv = s["q_start"].long(), s["kv_len"].long()
    n = q_start[1:] - q_start[:-1]
    T = s["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=T)
    pos = torch.arange(T, device=n.device) - q_start[seq] + (kv - n)[seq]
    P = s["case"]["page"]
    return seq, pos, s["table"].long()[seq, pos // P], pos % P


def _plain_append(s):
    c = s["case"]
    seq, pos, page, row = _token_places(s)
    cs = None if s["cos_sin"] is None else s["cos_sin"][pos]
    s["q_out"].copy_(_rotate(s["q"], cs, c["halves"]))
    _plain_store(s, "k", _rotate(s["k"], cs, c["halves"]), page, row)
    _plain_store(s, "v", s["v"].float(), page, row)
    return _append_outputs(s)


def _plain_store(s, name, x, page, row):
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        cache[page, :, row] = x.to(cache.dtype)
        return
    pages, Hkv, P, D = cache.shape
    amax = torch.zeros((pages, Hkv), device=x.device)
    amax.scatter_reduce_(0, page[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    fresh = torch.zeros(pages, dtype=torch.bool, device=x.device)
    fresh[page[row == 0]] = True                                  # the page's rows all come from this call
    old = scale.to(torch.int32) - 127
    new = old.clone()
    want = _exponent(amax)
    touched = torch.zeros(pages, dtype=torch.bool, device=x.device)
    touched[page] = True
    new = torch.where(touched[:, None], torch.where(fresh[:, None], want, torch.maximum(old, want)), old)
    codes = cache.view(torch.uint8)
    before = s["kv_len"].long() - torch.diff(s["q_start"].long())  # rows that each sequence held already
    kept = s["table"].long()[torch.arange(before.numel(), device=x.device), before // P]
    old_rows = torch.arange(P, device=x.device) < (before % P)[:, None]
    old_rows, kept = old_rows[~fresh[kept]], kept[~fresh[kept]]
    step = torch.exp2((old[kept] - new[kept]).double()).float()[:, :, None, None]
    again = (cache[kept].float() * step).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[kept] = torch.where((step < 1) & old_rows[:, None, :, None], again, codes[kept])
    inverse = torch.exp2(-new[page].double())[:, :, None]
    codes[page, :, row] = (x.double() * inverse).float().to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_((new + 127).to(torch.uint8))


def _rows(s, name, page, row):
    """Rows [B, L, Hkv, D] of a cache in float32."""
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        return cache[page, :, row].float()
    x = cache.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float()
    return x.mul_(torch.exp2(scale[page].float() - 127)[..., None])


def _plain_attend(s):
    c = s["case"]
    H, Hkv, D, P = c["H"], c["Hkv"], c["D"], c["page"]
    q_start, kv = s["q_start"].long(), s["kv_len"].long()
    B, N, L = kv.numel(), s["max_q"], s["max_kv"]
    dev = q_start.device
    n = (q_start[1:] - q_start[:-1])[:, None]
    i, j = torch.arange(N, device=dev)[None], torch.arange(L, device=dev)
    real = i < n
    token = (q_start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [B, N]
    pos = kv[:, None] - n + i
    page = s["table"].long()[:, (j // P)]
    row = (j % P).expand(B, -1)
    k, v = _rows(s, "k", page, row).permute(0, 2, 3, 1), _rows(s, "v", page, row).transpose(1, 2)
    q = s["q"][token].float().view(B, N, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    z = torch.matmul(q, k).view(B, Hkv, H // Hkv, N, L)
    z.mul_(s["scale"])
    if c["softcap"]:
        z.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    away = pos[:, :, None] - j
    if s["slopes"] is not None:
        z.addcmul_(s["slopes"].view(1, Hkv, -1, 1, 1), away.abs().float()[:, None, None], value=-1.0)
    see = (away >= 0) & (j < kv[:, None, None])
    if s["prefix_len"] is not None:
        see |= (j < torch.minimum(s["prefix_len"], s["kv_len"])[:, None, None])
    if c["window"]:
        see &= away < c["window"]
    if s["kv_start"] is not None:
        see &= j >= s["kv_start"][token][:, :, None]
    z.masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"].view(1, Hkv, -1, 1, 1))
    top = torch.where(top > -math.inf, top, 0.0)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True, dtype=torch.float64)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"].view(1, Hkv, -1, 1, 1) - top)
    o = torch.matmul(z.view(B, Hkv, -1, L), v).view(B, Hkv, -1, N, D)
    o = torch.where(total > 0, o / total, 0.0)
    s["out"][token[real]] = o.permute(0, 3, 1, 2, 4)[real].reshape(-1, H, D).to(torch.bfloat16)
    s["lse"][token[real]] = (top + torch.log(total)).permute(0, 3, 1, 2, 4)[real].reshape(-1, H).float()
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------
# the definition in float64, sequence by sequence
# ------------------------------------------------------------------------------------------------
def _e4m3(x):
    """x on the e4m3 grid (nearest, ties to even): 3 mantissa bits, smallest normal exponent -6."""
    _, e = torch.frexp(x)
    quantum = torch.exp2((e.double() - 1).clamp(min=-6.0) - 3)
    return torch.round(x / quantum) * quantum


def _exact_turn(x, angles_cos, angles_sin, first, halves):
    y = x.double().clone()
    half = angles_cos.shape[1]
    for d in range(half):
        i0, i1 = (first + d, first + half + d) if halves else (first + 2 * d, first + 2 * d + 1)
        a, b = x[:, :, i0].double(), x[:, :, i1].double()
        co, si = angles_cos[:, None, d].double(), angles_sin[:, None, d].double()
        y[:, :, i0] = a * co - b * si
        y[:, :, i1] = a * si + b * co
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    q_start, kv = s["q_start"].tolist(), s["kv_len"].tolist()
    G = case["H"] // case["Hkv"]
    for b in range(case["B"]):
        t0, t1 = q_start[b], q_start[b + 1]
        p = torch.arange(kv[b] - (t1 - t0), kv[b], device="cuda")[:, None]
        j = torch.arange(kv[b], device="cuda")[None]
        hidden = j > p
        if s["prefix_len"] is not None:
            hidden = hidden & (j >= int(s["prefix_len"][b]))
        if case["window"]:
            hidden = hidden | (j <= p - case["window"])
        if s["kv_start"] is not None:
            hidden = hidden | (j < s["kv_start"][t0:t1, None])
        where = s["table"][b, : -(-kv[b] // case["page"])].long()
        for h in range(case["Hkv"]):
            rows = []
            for name in ("k", "v"):
                x = s[name + "_cache"][where, h].double()
                if s[name + "_scale"] is not None:
                    x = x * torch.exp2(s[name + "_scale"][where, h].double() - 127)[:, None, None]
                rows.append(x.reshape(-1, case["D"])[: kv[b]])
            for a in range(h * G, h * G + G):
                z = s["q"][t0:t1, a].double() @ rows[0].T * s["scale"]
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][a].double() * (p - j).abs()
                z[hidden] = -math.inf
                if s["sink"] is not None:
                    z = torch.cat([z, s["sink"][a].double().expand(z.shape[0], 1)], 1)
                total = torch.logsumexp(z, 1)
                w = torch.exp(z[:, : kv[b]] - total.clamp(min=-1e300)[:, None])
                out[t0:t1, a] = w @ rows[1]
                lse[t0:t1, a] = total
    return {"out": out, "lse": lse}


def _exact_append(case, s):
    P, Hkv, half = case["page"], case["Hkv"], case["rope"] // 2
    q_start, kv = s["q_start"].tolist(), s["kv_len"].tolist()
    caches = {n: s[n + "_cache"].double() for n in ("k", "v")}
    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        t0, t1 = q_start[b], q_start[b + 1]
        p0 = kv[b] - (t1 - t0)
        turn = lambda x: x.double()  # noqa: E731
        if half:
            cs = s["cos_sin"][p0:kv[b]]
            turn = lambda x, cs=cs: _exact_turn(x, cs[:, :half], cs[:, half:], case["D"] - 2 * half, case["halves"])  # noqa: E731
        q[t0:t1] = turn(s["q"][t0:t1])
        for name, rows in (("k", turn(s["k"][t0:t1])), ("v", s["v"][t0:t1].double())):
            for first in range(p0 // P * P, kv[b], P):
                page = int(s["table"][b, first // P])
                lo, hi = max(first, p0), min(first + P, kv[b])
                new = rows[lo - p0:hi - p0].transpose(0, 1)           # [Hkv, rows, D]
                if s[name + "_scale"] is None:
                    caches[name][page, :, lo - first:hi - first] = new
                    continue
                amax = new.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / 448.0)).clamp(min=-127)
                e = torch.where(448.0 * torch.exp2(e - 1) >= amax, e - 1, e)
                e = torch.where(448.0 * torch.exp2(e) < amax, e + 1, e)
                e = torch.where(amax > 0, e, -127.0)
                if lo > first:
                    before = s[name + "_scale"][page].double() - 127
                    e = torch.maximum(e, before)
                    held = caches[name][page, :, :lo - first]
                    grown = _e4m3(held * torch.exp2(before - e)[:, None, None])
                    caches[name][page, :, :lo - first] = torch.where((e > before)[:, None, None], grown, held)
                caches[name][page, :, lo - first:hi - first] = _e4m3(new * torch.exp2(-e)[:, None, None])
    r = {"q": q, "k": caches["k"], "v": caches["v"]}
    if s["k_scale"] is not None:
        r.update(k_scale=None, v_scale=None)
    return r
