"""Measured cases of the operators around a decode step: rotary positions (rows turned, and the cos / sin tables that
the layers' calls take), the batch plan (pages, block tables, slot maps and positions from request lengths) and the
verification of drafted tokens.

`run` computes an operator in plain torch operations (float32, float64 for angles and next to a decision's border), or,
with `own` true, through the package's calls.  `exact` is the definition once more: float64 for the computed numbers,
integers request by request.

Definitions
rope    pair i of a head's rotated dims (2i, 2i + 1, or i, i + half) is turned by position * f_i and scaled; `inverse`
        turns back (the gradient of the forward turn).  f_i = theta^(-2i / dim), scaled for long contexts.
table   row p holds cos(p f_i) for every pair, then sin(p f_i).
plan    request b keeps ctx[b] + add[b] rows and brings n[b] tokens.  A cache stores floor(rows / ratio) entries in
        pages; the pages that a request no longer needs (behind its rows, or before its window) are pushed onto the
        cache's stack of free pages in order of the requests (of one request: front pages, then back pages), then
        missing pages are popped in order.  A request whose pages (or tokens) do not fit, counted over all requests up
        to it, gets no tokens in this step.
verify  token i of sequence b (i >= 1) was drafted from q_i; with p_i the target's probabilities after token i - 1 it
        stands if u q_i(x) < p_i(x) (greedy: if it is the target's first maximum).  The first one that falls is
        replaced by argmax_x max(p(x) - q(x), 0) / e(x), e given exponential variates; when all stand one more token
        argmax_x p(x) / e(x) follows.
"""
import math

import numpy as np
import torch

own = False

_ROPE = {"op": "rope", "T": 1, "H": 64, "Hkv": 8, "D": 128, "rope": 128, "first": 0, "halves": False, "inverse": False,
         "dtype": "bf16", "far": 4096, "theta": 10000.0, "scaling": "none", "factor": 1.0, "orig": 4096, "scale": 1.0}
_TABLE = {"op": "table", "rows": 4096, "rope": 64, "theta": 10000.0, "scaling": "none", "factor": 1.0, "orig": 4096,
          "scale": 1.0}
# caches: "page:ratio:window" of each, separated by blanks
_PLAN = {"op": "plan", "B": 1, "n": 1, "n_spread": 0.0, "ctx": 1000, "spread": 0.9, "caches": "64:1:0", "spare": 1.3,
         "ended": 0.05}
_VERIFY = {"op": "verify", "B": 1, "n": 4, "n_spread": 0.0, "V": 32000, "target": "bf16", "draft": "bf16",
           "target_probs": False, "draft_probs": False, "greedy": 0.0, "temp": 0.8, "banned": 0.0}


def _case(base, **kw):
    c = dict(base)
    c.update(kw)
    return c


def listed():
    return [
        # queries and keys of one decode step of 12 sequences with four tokens each, context scaled eightfold
        _case(_ROPE, name="rope_step_48", T=48, far=32768, scaling="yarn", factor=8.0, scale=1.2079),
        # ragged prompts of a small layer: part of a 64-wide head, halves, rows of a fused projection
        _case(_ROPE, name="rope_prompt_halves", T=9377, H=20, Hkv=4, D=64, rope=32, first=32, halves=True, far=9000),
        # gradient of the queries' rotation in a training step, float32
        _case(_ROPE, name="rope_back_fp32", T=4096, H=32, Hkv=0, dtype="fp32", inverse=True, theta=500000.0),
        # a large prompt chunk far into a context of a million rows
        _case(_ROPE, name="rope_prompt_16k", T=16384, far=1 << 20, scaling="yarn", factor=32.0, orig=32768, scale=1.3466),
        # the table that the layers' calls take, for a context of 128k rows
        _case(_TABLE, name="rope_table_128k", rows=131072, rope=64, scaling="bands", factor=8.0, orig=8192),
        # a decode step of 64 requests with four tokens each over one cache
        _case(_PLAN, name="plan_step_64", B=64, n=4, ctx=4000),
        # a large decode step of a hybrid layer: window, one entry for 4 rows and one for 128; pages are short
        _case(_PLAN, name="plan_step_1000_hybrid", B=1000, n=4, n_spread=0.8, ctx=20000,
              caches="64:1:128 64:4:0 64:128:0", spare=0.02),
        # prompts beside decode steps, small pages
        _case(_PLAN, name="plan_prompts_64k", B=300, n=440, n_spread=0.99, ctx=2000, caches="16:1:0"),
        # the smallest call: two sequences, logits of both models in float32
        _case(_VERIFY, name="verify_2x4_32k", B=2, V=32000, target="fp32", draft="fp32"),
        # a serving batch; the drafter kept the probabilities it drew from
        _case(_VERIFY, name="verify_64x4_128k", B=64, V=131072, draft="fp32", draft_probs=True, banned=0.1),
        # drafts looked up in the text (no probabilities), half of the requests greedy, odd vocabulary
        _case(_VERIFY, name="verify_200x3_odd", B=200, n=3, n_spread=0.7, V=100003, draft="none", greedy=0.5),
        # a large batch, logits of both models
        _case(_VERIFY, name="verify_256x5_128k", B=256, n=5, V=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_scaling(rng):
    kind = rng.choice(["none", "linear", "base", "yarn", "bands"])
    factor = 1.0 if kind == "none" else rng.choice([2.0, 8.0, 40.0])
    return {"scaling": kind, "factor": factor, "orig": rng.choice([2048, 4096, 8192]),
            "theta": rng.choice([10000.0, 160000.0, 1000000.0]), "scale": rng.choice([1.0, 1.0, 1.25])}


def draw(rng):
    op = rng.choice(["rope", "rope", "table", "plan", "plan", "verify", "verify", "verify"])
    if op == "table":
        rope = rng.choice([32, 64, 96, 128])
        return _case(_TABLE, rows=_log(rng, 100, 131072 * 64 // rope), rope=rope, **_draw_scaling(rng))
    if op == "rope":
        D = rng.choice([64, 80, 128, 128, 192, 256])
        rope = rng.choice([D, D // 32 * 16, 32])
        Hkv = rng.choice([0, 1, 2, 8])
        H = rng.choice([1, 5, 12, 32, 64])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = 16384 * 72 * 128 // ((H + Hkv) * D * (2 if dtype == "fp32" else 1))
        return _case(_ROPE, T=_log(rng, 1, min(16384, most)), H=H, Hkv=Hkv, D=D, rope=rope, dtype=dtype,
                     first=rng.choice([0, D - rope]), halves=rng.random() < 0.5, inverse=rng.random() < 0.3,
                     far=_log(rng, 1000, 1 << 20), **_draw_scaling(rng))
    if op == "plan":
        n = rng.choice([1, 2, 4, _log(rng, 5, 3000)])
        B = _log(rng, 1, min(4000, 131072 // n))
        return _case(_PLAN, B=B, n=n, n_spread=rng.choice([0.0, 0.9]), ctx=_log(rng, 1, 30000),
                     spread=rng.choice([0.0, 0.9]), spare=rng.choice([0.05, 1.2]), ended=rng.choice([0.0, 0.1]),
                     caches=rng.choice(["64:1:0", "16:1:0", "32:1:500", "64:1:128 64:4:0", "128:1:0 256:4:0 64:128:0"]))
    V = _log(rng, 1000, 150000)
    n = rng.choice([1, 2, 3, 4, 5, 8])
    draft = rng.choice(["none", "bf16", "bf16", "fp32", "fp32"])
    return _case(_VERIFY, B=_log(rng, 1, min(512, max(1, 1280 * 131072 // (2 * n * V)))), n=n,
                 n_spread=rng.choice([0.0, 0.8]), V=V, target=rng.choice(["bf16", "bf16", "fp32"]), draft=draft,
                 target_probs=rng.random() < 0.2, draft_probs=draft == "fp32" and rng.random() < 0.6,
                 greedy=rng.choice([0.0, 0.0, 0.3]), temp=rng.choice([0.5, 0.8, 1.0]), banned=rng.choice([0.0, 0.2]))


def _lens(B, top, spread):
    """Ragged lengths: the first is `top`, the others lie between top * (1 - spread) and top."""
    return np.floor(top * (1.0 - spread * np.mod(np.arange(B) * 0.6180339887, 1.0))).astype(np.int64)


_KEPT = 0.75  # a drafted token of these inputs stands in about three cases of four


def work(case):
    c = case
    if c["op"] == "rope":
        elements = c["T"] * (c["H"] + c["Hkv"]) * c["D"]
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2 * size * elements + 4 * c["T"], "flops": 3 * elements * c["rope"] // c["D"]}
    if c["op"] == "table":
        return {"bytes": 4 * c["rows"] * c["rope"], "flops": 20 * c["rows"] * c["rope"]}
    if c["op"] == "plan":
        T = int(np.maximum(1, _lens(c["B"], c["n"], c["n_spread"])).sum())
        caches = len(c["caches"].split())
        return {"bytes": c["B"] * (12 + 8 + 8 * caches) + T * (8 + 8 * caches), "flops": 4 * T * caches}
    n = np.maximum(1, _lens(c["B"], c["n"], c["n_spread"]))
    V = c["V"]
    rows = float(sum((1 - _KEPT ** int(k)) / (1 - _KEPT) for k in n))      # up to the first token that falls
    drafted = float(sum((1 - _KEPT ** (int(k) - 1)) / (1 - _KEPT) for k in n))
    fallen = float(sum(1 - _KEPT ** (int(k) - 1) for k in n))
    size = lambda kind: 4 if kind == "fp32" else 2  # noqa: E731
    b = V * size(c["target"]) * (c["B"] if c["target_probs"] else rows)
    if c["draft"] != "none":
        b += V * size(c["draft"]) * (fallen if c["draft_probs"] else drafted) * (1 - c["greedy"])
    b += 4 * V * c["B"] * (1 - c["greedy"])
    return {"bytes": int(b), "flops": int(4 * V * (rows + c["B"]))}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _frequencies(c):
    """f_i of every pair in radians a position, float64 (numpy)."""
    dim, theta, factor = c["rope"], c["theta"], c["factor"]
    i = np.arange(dim // 2, dtype=np.float64)
    if c["scaling"] == "base":
        theta = theta * factor ** (dim / (dim - 2))
    f = theta ** (-2.0 * i / dim)
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "yarn":
        turns = lambda r: dim * math.log(c["orig"] / (r * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), dim - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f / factor * ramp + f * (1 - ramp)
    elif c["scaling"] == "bands":
        wave = 2 * math.pi / f
        mix = np.clip((c["orig"] / wave - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = (1 - mix) * f / factor + mix * f
    return f


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "table": _prepare_table, "plan": _prepare_plan,
            "verify": _prepare_verify}[case["op"]](case, g, seed)


def _prepare_rope(c, g, seed):
    T, H, Hkv, D = c["T"], c["H"], c["Hkv"], c["D"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    qkv = torch.randn((T, H + 2 * Hkv, D), generator=g, device="cuda").to(dt)   # rows of one fused projection
    # each token at its own place of the context (packed sequences)
    pos = torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    s = {"case": c, "q": qkv[:, :H], "k": qkv[:, H:H + Hkv] if Hkv else None, "pos": pos,
         "freq": torch.from_numpy(_frequencies(c)).cuda(), "q_out": torch.empty((T, H, D), dtype=dt, device="cuda")}
    s["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda") if Hkv else None
    return s


def _prepare_table(c, g, seed):
    first = int(torch.randint(0, 5000, (1,), generator=g, device="cuda"))
    return {"case": c, "first": first, "freq": torch.from_numpy(_frequencies(c)).cuda(),
            "table": torch.empty((c["rows"], c["rope"]), dtype=torch.float32, device="cuda")}


def _prepare_plan(c, g, seed):
    r = np.random.default_rng(seed)
    B = c["B"]
    n = r.permutation(np.maximum(1, _lens(B, c["n"], c["n_spread"])))
    T = -(-int(n.sum()) // 64) * 64                    # a captured step's token count: padded
    before = r.permutation(_lens(B, c["ctx"], c["spread"]))
    most = np.sort(before) + 8 + int(n.max())          # rows that a request of this batch can come to
    standing = before.copy()
    add = r.integers(0, 5, B)                          # what the last step's verification let stand
    waiting = r.random(B) < 0.05                       # requests that begin in this step
    before[waiting], add[waiting] = 0, 0
    ended = r.random(B) < c["ended"]
    before[ended], add[ended], n[ended] = 0, 0, 0
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.int32)  # noqa: E731
    s = {"case": c, "ctx": ints(before), "add": ints(add), "n": ints(n), "T": T, "caches": []}
    new = lambda *shape, dt=torch.int32: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    for text in c["caches"].split():
        P, ratio, window = (int(x) for x in text.split(":"))
        # rows held when the last step began: up to four more than stood; an ended request still holds its pages
        rows = np.where(waiting, 0, before + add + r.integers(0, 4, B))
        rows = np.where(ended, standing, rows)
        held = -(-(rows // ratio) // P)
        first = np.zeros(B, np.int64)
        if window:
            first = np.where(ended | waiting, 0, np.minimum(held, np.maximum(0, before - window + 1) // P))
        missing = int(np.maximum(0, -(-((before + add + n) // ratio) // P) - held).sum())
        used = held - first
        pages, width = int((-(-(most // ratio) // P) + 1).sum()), int(-(-(most.max() // ratio) // P) + 1)
        free = min(int(missing * c["spare"]) + 2, pages - int(used.sum()))
        order = r.permutation(pages)
        table = np.full((B, width), -1, np.int64)
        cols = np.arange(width)[None]
        table[(cols >= first[:, None]) & (cols < held[:, None])] = order[free:free + int(used.sum())]
        stack = np.full(pages, -1, np.int64)
        stack[:free] = order[:free]
        s["caches"].append({
            "page": P, "ratio": ratio, "window": window, "table": ints(table), "held": ints(held), "first": ints(first),
            "stack": ints(stack), "count": ints(np.array([free])), "held_out": new(B), "first_out": new(B),
            "count_out": new(1), "slots": new(T, dt=torch.int64)})
    s.update(ctx_out=new(B), q_start=new(B + 1), kv_len=new(B), pos=new(T), seq=new(T))
    return s


def _prepare_verify(c, g, seed):
    B, V = c["B"], c["V"]
    n = np.maximum(1, _lens(B, c["n"], c["n_spread"]))
    start = np.concatenate([[0], np.cumsum(n)])
    T, D = int(start[-1]), int(start[-1]) - B
    dtype = {"bf16": torch.bfloat16, "fp32": torch.float32, "none": torch.float32}
    dev = "cuda"
    seq = torch.from_numpy(np.repeat(np.arange(B), n)).to(dev)
    greedy = torch.from_numpy(np.mod(np.arange(B) * 0.754877, 1.0) < c["greedy"]).to(dev)
    temp = torch.full((B,), c["temp"], device=dev) * (0.8 + 0.4 * torch.rand((B,), generator=g, device=dev))
    temp[greedy] = 0.0
    soft = torch.where(greedy, 1.0, temp)
    target = torch.empty((T, V), dtype=dtype[c["target"]], device=dev)
    draft = torch.empty((max(D, 1), V), dtype=dtype[c["draft"]], device=dev) if c["draft"] != "none" else None
    tokens = torch.randint(0, V, (T,), generator=g, device=dev, dtype=torch.int32)
    heads = np.zeros(T, bool)
    heads[start[:-1]] = True
    follows = torch.from_numpy(~np.append(heads[1:], True)).to(dev)        # row t has a drafted successor
    rows = max(1, (1 << 25) // V)
    for t0 in range(0, T, rows):
        t1 = min(T, t0 + rows)
        m = t1 - t0
        # a few words that fit, far above the rest; a drafter that mostly agrees
        z = torch.randn((m, V), generator=g, device=dev).mul_(2.0)
        top = torch.randint(0, V, (m, 12), generator=g, device=dev)
        z.scatter_(1, top, 8.0 + 3.0 * torch.randn((m, 12), generator=g, device=dev))
        y = z + 0.35 * torch.randn((m, V), generator=g, device=dev)
        if c["banned"]:
            z.masked_fill_(torch.rand((m, V), generator=g, device=dev) < c["banned"], -math.inf)
        z, y = z.to(target.dtype), y.to(dtype[c["draft"]])
        t = soft[seq[t0:t1]][:, None]
        if c["target_probs"]:
            target[t0:t1] = torch.softmax(z.float() / t, 1).to(target.dtype)
        else:
            target[t0:t1] = z
        q = torch.softmax(y.float() / t, 1)
        drawn = (q / torch.empty_like(q).exponential_(generator=g)).argmax(1)
        best = y.float().argmax(1)
        drawn = torch.where(greedy[seq[t0:t1]], best, drawn)
        here = torch.arange(t0, t1, device=dev)[follows[t0:t1]]
        tokens[here + 1] = drawn[follows[t0:t1]].to(torch.int32)
        if draft is not None and len(here):
            draft[here - seq[here]] = (q if c["draft_probs"] else y)[follows[t0:t1]].to(draft.dtype)
    noise = torch.empty((B, V), device=dev)
    for b0 in range(0, B, rows):
        noise[b0:b0 + rows].exponential_(generator=g).clamp_(min=1e-30)
    W = int(n.max())
    return {"case": c, "target": target, "draft": draft, "tokens": tokens, "temp": temp, "noise": noise, "W": W,
            "u": torch.rand((T,), generator=g, device=dev),
            "q_start": torch.from_numpy(start).to(dev).to(torch.int32),
            "out": torch.empty((B, W), dtype=torch.int32, device=dev),
            "count": torch.empty((B,), dtype=torch.int32, device=dev),
            "logp": torch.empty((B, W), dtype=torch.float32, device=dev)}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "table": _own_table, "plan": _own_plan, "verify": _own_verify}[op](s)
    return {"rope": _plain_rope, "table": _plain_table, "plan": _plain_plan, "verify": _plain_verify}[op](s)


# ------------------------------------------------------------------------------------------------
# the package's calls.  As in a decode loop over fixed buffers, a call's parameters are filled in on
# the first pass over a state and kept beside its buffers.
# ------------------------------------------------------------------------------------------------
def _own_freqs(M, c):
    return M.rope_freqs(c["rope"], theta=c["theta"], scaling=c["scaling"], factor=c["factor"], original_len=c["orig"],
                        beta_fast=32.0, beta_slow=1.0, low_turns=1.0, high_turns=4.0, device="cuda")


def _own_rope(s):
    import deepseek_v4_hybrid_gb300 as M
    if "plan" not in s:
        c = s["case"]
        s["plan"] = M.rope_params(s["q"], s["q_out"], s["pos"], _own_freqs(M, c), x2=s["k"], out2=s["k_out"],
                                  rope_first=c["first"], rope_halves=c["halves"], inverse=c["inverse"], scale=c["scale"])
    M.dsv4_rope(s["plan"])
    return {"q": s["q_out"], "k": s["k_out"]} if s["k"] is not None else {"q": s["q_out"]}


def _own_table(s):
    import deepseek_v4_hybrid_gb300 as M
    if "plan" not in s:
        s["plan"] = M.rope_table_params(s["table"], _own_freqs(M, s["case"]), first_position=s["first"],
                                        scale=s["case"]["scale"])
    M.dsv4_rope_table(s["plan"])
    return s["table"]


def _own_plan(s):
    import deepseek_v4_hybrid_gb300 as M
    if "plan" not in s:
        caches = [M.plan_cache(k["table"], k["held"], k["stack"], k["count"], k["page"], held_out=k["held_out"],
                               free_count_out=k["count_out"], ratio=k["ratio"], window=k["window"],
                               first=k["first"] if k["window"] else None,
                               first_out=k["first_out"] if k["window"] else None, slots=k["slots"])
                  for k in s["caches"]]
        s["plan"] = M.batch_plan_params(s["ctx"], s["n"], s["q_start"], s["kv_len"], caches, ctx_add=s["add"],
                                        ctx_out=s["ctx_out"], positions=s["pos"], token_seq=s["seq"])
    M.dsv4_batch_plan(s["plan"])
    return _plan_outputs(s)


def _own_verify(s):
    import deepseek_v4_hybrid_gb300 as M
    if "plan" not in s:
        c = s["case"]
        s["plan"] = M.draft_verify_params(
            s["target"], s["tokens"], s["q_start"], s["W"], s["out"], s["count"], draft=s["draft"],
            temperature=s["temp"], u=s["u"], noise=s["noise"], logp=s["logp"], target_probs=c["target_probs"],
            draft_probs=c["draft_probs"])
    M.dsv4_draft_verify(s["plan"])
    return {"tokens": s["out"], "count": s["count"], "logp": s["logp"]}


def _plan_outputs(s):
    r = {k: s[k] for k in ("ctx_out", "q_start", "kv_len", "pos", "seq")}
    for i, k in enumerate(s["caches"]):
        for name in ("table", "held_out", "stack", "count_out", "slots") + (("first_out",) if k["window"] else ()):
            r[f"{name}{i}"] = k[name]
    return r


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _plain_turn(x, out, cos, sin, c):
    half, first = c["rope"] // 2, c["first"]
    y = x.float().clone()
    part = y[..., first:first + c["rope"]]
    a, b = (part[..., :half], part[..., half:]) if c["halves"] else (part[..., 0::2], part[..., 1::2])
    turned = (a * cos - b * sin, b * cos + a * sin)
    if c["halves"]:
        y[..., first:first + half], y[..., first + half:first + c["rope"]] = turned
    else:
        y[..., first:first + c["rope"]:2], y[..., first + 1:first + c["rope"]:2] = turned
    out.copy_(y)


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (angle.cos() * c["scale"]).float()[:, None], (angle.sin() * c["scale"]).float()[:, None]
    if c["inverse"]:
        sin = -sin
    _plain_turn(s["q"], s["q_out"], cos, sin, c)
    if s["k"] is None:
        return {"q": s["q_out"]}
    _plain_turn(s["k"], s["k_out"], cos, sin, c)
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_table(s):
    c = s["case"]
    p = torch.arange(s["first"], s["first"] + c["rows"], dtype=torch.float64, device="cuda")
    angle = p[:, None] * s["freq"]
    s["table"].copy_(torch.cat([angle.cos(), angle.sin()], 1) * c["scale"])
    return s["table"]


def _before(x):
    """Sums of the entries before each one."""
    return torch.cumsum(x, 0) - x


def _plain_plan(s):
    dev = s["n"].device
    n, ctx = s["n"].long(), s["ctx"].long() + s["add"].long()
    B, T = n.numel(), s["T"]
    b = torch.arange(B, device=dev)
    runs = (n == 0) | (torch.cumsum(n, 0) <= T)
    todo = []
    for k in s["caches"]:
        held, first, P = k["held"].long(), k["first"].long(), k["page"]
        need = ((ctx + n) // k["ratio"] + P - 1) // P
        lo = first
        if k["window"]:
            lo = torch.minimum(held, torch.maximum(first, (ctx - k["window"] + 1).clamp(min=0) // P))
        over = ctx + n == 0
        keep = torch.where(over, first, torch.maximum(need, lo))
        front, back = torch.where(over, 0, lo - first), (held - keep).clamp(min=0)
        take = (need - held).clamp(min=0)
        count = k["count"].long()
        # given back: front pages, then back pages of each request
        given = front + back
        at = _before(given)
        col = torch.arange(k["table"].shape[1], device=dev)[None]
        is_front = (col >= first[:, None]) & (col < (first + front)[:, None])
        is_back = (col >= (held - back)[:, None]) & (col < held[:, None])
        place = torch.where(is_front, col - first[:, None], col - (held - back - front)[:, None]) + (count + at)[:, None]
        room = k["stack"].numel()
        pushed = torch.cat([k["stack"].long(), torch.zeros(1, dtype=torch.long, device=dev)])
        pushed.scatter_(0, torch.where(is_front | is_back, place, room).flatten(), k["table"].long().flatten())
        k["stack"].copy_(pushed[:room])
        top = count + given.sum()
        runs = runs & ((take == 0) | (torch.cumsum(take, 0) <= top))
        todo.append((k, held, first, lo, front, back, over, take, top, col, need))
    n = torch.where(runs, n, 0)
    for k, held, first, lo, front, back, over, take, top, col, need in todo:
        take = torch.where(runs, take, 0)
        new = (col >= held[:, None]) & (col < (held + take)[:, None])
        source = (top - 1 - _before(take))[:, None] - (col - held[:, None])
        k["table"].copy_(torch.where(new, k["stack"][source.clamp(0, k["stack"].numel() - 1)], k["table"]))
        k["held_out"].copy_(torch.where(over, 0, held - back + take))
        k["first_out"].copy_(torch.where(over, 0, lo))
        k["count_out"].copy_(top - take.sum())
    end = torch.cumsum(n, 0)
    s["ctx_out"].copy_(ctx)
    s["kv_len"].copy_(ctx + n)
    s["q_start"][0] = 0
    s["q_start"][1:] = end
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(end, t, right=True)
    real = seq < B
    seq = seq.clamp(max=B - 1)
    pos = t - (end - n)[seq] + ctx[seq]
    s["pos"].copy_(torch.where(real, pos, -1))
    s["seq"].copy_(torch.where(real, seq, -1))
    for k in s["caches"]:
        P, r = k["page"], k["ratio"]
        entry = pos // r
        page = k["table"].long()[seq, (entry // P).clamp(0, k["table"].shape[1] - 1)]
        stored = real & ((pos + 1) % r == 0)
        k["slots"].copy_(torch.where(stored, page * P + entry % P, -1))
    return _plan_outputs(s)


def _plain_weights(rows, probs, soft):
    """e^(z / T - max), the maximum and the sum of every row (probabilities: as they are, 0 and 1)."""
    x = rows.float()
    if probs:
        return x, torch.zeros(x.shape[0], device=x.device), torch.ones(x.shape[0], dtype=torch.float64, device=x.device)
    top = x.amax(1)
    w = torch.exp((x - top[:, None]) / soft[:, None])
    return w, top, w.sum(1, dtype=torch.float64)


def _plain_prob(rows, index, token, probs, top, total, soft):
    """Probability of one token of each row and its logarithm, float64 (its weight lies next to a border)."""
    x = rows[index, token].double()
    if probs:
        return x, torch.log(x)
    a = (x - top.double()[index]) / soft
    return torch.exp(a) / total[index], a - torch.log(total[index])


def _plain_verify(s):
    c = s["case"]
    dev, W, V = s["target"].device, s["W"], c["V"]
    T = s["target"].shape[0]
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    B = n.numel()
    greedy = s["temp"] <= 0
    soft = torch.where(greedy, 1.0, s["temp"]).double()
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(start[1:], t, right=True)
    _, top, total = _plain_weights(s["target"], c["target_probs"], soft[seq].float())
    x = s["target"].float()
    best = torch.where(x == x.amax(1, keepdim=True), torch.arange(V, device=dev), V).amin(1)
    i = torch.arange(W, device=dev)[None]
    row = (start[:-1, None] + i).clamp(max=T - 1)                       # [B, W] row i of each sequence
    nxt = (row + 1).clamp(max=T - 1)
    drafted = i < n[:, None] - 1
    token = s["tokens"].long()[nxt]
    softb = soft[:, None].expand(B, W)
    p, logp = _plain_prob(s["target"], row, token, c["target_probs"], top, total, softb)
    if s["draft"] is None:
        stands = s["u"].double()[nxt] < p
    else:
        drow = (row - torch.arange(B, device=dev)[:, None]).clamp(max=s["draft"].shape[0] - 1)
        drawn_before = (start[1:] - torch.arange(1, B + 1, device=dev)).contiguous()
        dseq = torch.searchsorted(drawn_before, torch.arange(s["draft"].shape[0], device=dev), right=True).clamp(max=B - 1)
        _, dtop, dtotal = _plain_weights(s["draft"], c["draft_probs"], soft[dseq].float())
        q, _ = _plain_prob(s["draft"], drow, token, c["draft_probs"], dtop, dtotal, softb)
        stands = s["u"].double()[nxt] * q < p
    stands = torch.where(greedy[:, None], token == best[row], stands) & drafted
    kept = torch.cumprod(stands.long(), 1).sum(1)                       # drafted tokens that stand
    all_stand = kept == n - 1
    b = torch.arange(B, device=dev)
    last = start[:-1] + kept                                            # the row that the last token comes from
    w = _plain_last(s["target"], last, c["target_probs"], top, total, soft)
    r = w
    fell = s["tokens"].long()[(last + 1).clamp(max=T - 1)]
    if s["draft"] is None:
        r = torch.where((torch.arange(V, device=dev)[None] == fell[:, None]) & ~all_stand[:, None], 0.0, w)
    else:
        d = _plain_last(s["draft"], (last - b).clamp(max=s["draft"].shape[0] - 1), c["draft_probs"], dtop, dtotal, soft)
        r = torch.where(all_stand[:, None], w, (w - d).clamp(min=0))
    r = torch.where(r.amax(1, keepdim=True) > 0, r, w)
    chosen = torch.where(greedy, best[last], (r / s["noise"]).argmax(1))
    _, last_logp = _plain_prob(s["target"], last, chosen, c["target_probs"], top, total, soft)
    out = torch.where(i < kept[:, None], token, -1)
    out[b, kept] = chosen
    lp = torch.where(i < kept[:, None], logp, 0.0)
    lp[b, kept] = last_logp
    s["out"].copy_(out)
    s["count"].copy_(kept + 1)
    s["logp"].copy_(lp)
    return {"tokens": s["out"], "count": s["count"], "logp": s["logp"]}


def _plain_last(rows, index, probs, top, total, soft):
    """Probabilities of one row for each sequence, float64."""
    x = rows[index].double()
    if probs:
        return x
    return torch.exp((x - top.double()[index][:, None]) / soft[:, None]) / total[index][:, None]


# ------------------------------------------------------------------------------------------------
# the definitions once more
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "table": _exact_table, "plan": _exact_plan, "verify": _exact_verify}[case["op"]](case, s)


def _exact_rope(c, s):
    half = c["rope"] // 2
    sign = -1.0 if c["inverse"] else 1.0

    def turned(x):
        y = x.double()
        for i in range(half):
            i0, i1 = (i, half + i) if c["halves"] else (2 * i, 2 * i + 1)
            i0, i1 = i0 + c["first"], i1 + c["first"]
            angle = s["pos"].double() * s["freq"][i]
            z = torch.complex(x[:, :, i0].double(), x[:, :, i1].double())
            z = z * torch.polar(torch.full_like(angle, c["scale"]), sign * angle)[:, None]
            y[:, :, i0], y[:, :, i1] = z.real, z.imag
        return y

    r = {"q": turned(s["q"])}
    if s["k"] is not None:
        r["k"] = turned(s["k"])
    return r


def _exact_table(c, s):
    rows = torch.arange(c["rows"], device="cuda").double() + s["first"]
    out = torch.empty((c["rows"], c["rope"]), dtype=torch.float64, device="cuda")
    for i in range(c["rope"] // 2):
        out[:, i] = torch.cos(rows * s["freq"][i]) * c["scale"]
        out[:, c["rope"] // 2 + i] = torch.sin(rows * s["freq"][i]) * c["scale"]
    return out


def _exact_plan(c, s):
    B, T = c["B"], s["T"]
    ctx = [x + y for x, y in zip(s["ctx"].tolist(), s["add"].tolist())]
    n = s["n"].tolist()
    pools, runs, total = [], [True] * B, 0
    for b in range(B):
        total += n[b]
        runs[b] = n[b] == 0 or total <= T
    for k in s["caches"]:
        stack = k["stack"].tolist()
        tab, held, first = k["table"].tolist(), k["held"].tolist(), k["first"].tolist()
        level = k["count"].item()
        need = [-(-((ctx[b] + n[b]) // k["ratio"]) // k["page"]) for b in range(B)]
        held_before = list(held)
        for b in range(B):
            if ctx[b] + n[b] == 0:
                gone, lo, hi = list(range(first[b], held[b])), 0, 0
            else:
                lo = first[b]
                if k["window"]:
                    lo = min(held[b], max(lo, max(0, ctx[b] - k["window"] + 1) // k["page"]))
                hi = min(held[b], max(need[b], lo))
                gone = list(range(first[b], lo)) + list(range(hi, held[b]))
            for j in gone:
                stack[level] = tab[b][j]
                level += 1
            first[b], held[b] = lo, hi
        wanted = 0
        for b in range(B):
            take = max(0, need[b] - held_before[b])
            wanted += take
            if take and wanted > level:
                runs[b] = False
        pools.append([k, stack, tab, held, first, level, need, held_before])
    for pool in pools:
        k, stack, tab, held, first, level, need, held_before = pool
        for b in range(B):
            for j in range(held_before[b], need[b]):
                if runs[b]:
                    level -= 1
                    tab[b][j] = stack[level]
                    held[b] = j + 1
        pool[5] = level
    n = [x if r else 0 for x, r in zip(n, runs)]
    pos, seq = [], []
    for b in range(B):
        pos += range(ctx[b], ctx[b] + n[b])
        seq += [b] * n[b]
    pad = [-1] * (T - len(pos))
    as_ints = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    r = {"ctx_out": as_ints(ctx), "q_start": as_ints([0] + list(np.cumsum(n))),
         "kv_len": as_ints([x + y for x, y in zip(ctx, n)]), "pos": as_ints(pos + pad), "seq": as_ints(seq + pad)}
    for i, (k, stack, tab, held, first, level, _, _) in enumerate(pools):
        slots = []
        for p, b in zip(pos, seq):
            e = p // k["ratio"]
            slots.append(tab[b][e // k["page"]] * k["page"] + e % k["page"] if (p + 1) % k["ratio"] == 0 else -1)
        r.update({f"table{i}": as_ints(tab), f"held_out{i}": as_ints(held), f"stack{i}": as_ints(stack),
                  f"count_out{i}": as_ints([level]), f"slots{i}": as_ints(slots + pad)})
        if k["window"]:
            r[f"first_out{i}"] = as_ints(first)
    return r


def _exact_verify(c, s):
    B, W = c["B"], s["W"]
    start, tokens = s["q_start"].tolist(), s["tokens"].tolist()
    temp, u = s["temp"].double().tolist(), s["u"].double().tolist()
    out = torch.full((B, W), -1, dtype=torch.int64)
    logp = torch.zeros((B, W), dtype=torch.float64)
    count = torch.zeros(B, dtype=torch.int64)

    def law(row, probs, T):
        x = row.double()
        return (x, torch.log(x)) if probs else (torch.softmax(x / T, 0), torch.log_softmax(x / T, 0))

    for b in range(B):
        n, T = start[b + 1] - start[b], temp[b]
        for i in range(n):
            t = start[b] + i
            p, lp = law(s["target"][t], c["target_probs"], T if T > 0 else 1.0)
            first_best = int(torch.nonzero(s["target"][t] == s["target"][t].max())[0])
            x = tokens[t + 1] if i + 1 < n else -1
            left = p
            if x >= 0:
                if T <= 0:
                    ok = x == first_best
                elif s["draft"] is None:
                    ok = u[t + 1] < float(p[x])
                    left = p.clone()
                    left[x] = 0
                else:
                    q, _ = law(s["draft"][t - b], c["draft_probs"], T)
                    ok = u[t + 1] * float(q[x]) < float(p[x])
                    left = torch.clamp(p - q, min=0)
                if ok:
                    out[b, i], logp[b, i] = x, lp[x]
                    continue
            if float(left.max()) <= 0:
                left = p
            y = first_best if T <= 0 else int(torch.argmax(left / s["noise"][b].double()))
            out[b, i], logp[b, i], count[b] = y, lp[y], i + 1
            break
    return {"tokens": out.cuda(), "count": count.cuda(), "logp": logp.cuda()}
