"""The calls around the layers on the GPU against their float64 and integer definitions."""
import math

import numpy as np
import pytest
import torch

from oracle import loop_oracle as L

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_v4_hybrid_gb300 as mod
    return mod


def f64(t):
    return t.double().cpu().numpy()


def ints(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


# ------------------------------------------------------------------------------------------------
# rotary positions
# ------------------------------------------------------------------------------------------------
def rope_bound(x, want, first, dim, halves, scale, dtype):
    """An angle's float conversion moves it by pi 2^-24 at most, the sums for sine and cosine by two steps of 2^-24, the
    factor's product by half a step; two products and a sum round once or twice each: |a| and |b| times 8 * 2^-24 in all.
    Then the output's rounding; dims that are copied are exact."""
    a = np.abs(x).copy()
    part = a[:, :, first:first + dim]
    pair = part.reshape(*part.shape[:2], 2, -1).sum(2) if halves else part.reshape(*part.shape[:2], -1, 2).sum(3)
    size = np.concatenate([pair, pair], 2) if halves else np.repeat(pair, 2, 2)
    tol = np.zeros_like(a)
    tol[:, :, first:first + dim] = abs(scale) * size * 8 * 2.0 ** -24 + 1e-37
    if dtype == BF16:
        tol[:, :, first:first + dim] += 2.0 ** -8 * (np.abs(want)[:, :, first:first + dim] +
                                                     tol[:, :, first:first + dim])
    return tol


ROPES = [  # T, heads, heads2, dim, first, rope_dim, halves
    (1, 1, 0, 16, 0, 16, False), (1, 64, 8, 128, 0, 128, False), (3, 5, 1, 64, 32, 32, True), (70, 20, 4, 64, 0, 64, True),
    (33, 7, 3, 80, 48, 32, False), (129, 1, 0, 576, 512, 64, False), (5, 3, 2, 1024, 0, 1024, True),
    (9, 128, 1, 192, 128, 64, False), (1000, 1, 1, 256, 8, 48, True), (17, 300, 0, 96, 0, 96, False),
    (40, 2, 2, 24, 8, 16, True), (3, 2, 0, 1024, 0, 1024, False), (2, 1024, 1, 32, 0, 32, False),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", ROPES, ids=lambda s: "_".join(str(int(x)) for x in s))
def test_rope(M, shape, dtype):
    T, H, H2, D, first, dim, halves = shape
    g = torch.Generator(device="cuda").manual_seed(T * H + D)
    fused = torch.randn((T, H + 2 * H2 + 1, D), generator=g, device="cuda").to(dtype)
    x, x2 = fused[:, :H], fused[:, H:H + H2] if H2 else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -1
    freqs = M.rope_freqs(dim, scaling="yarn", factor=8.0, original_len=4096)
    hf = freqs.cpu().numpy()
    scale, before = 1.25, fused.clone()
    live = (pos >= 0).cpu().numpy()
    for inverse in (False, True):
        for place in ("apart", "in place"):
            fused.copy_(before)
            src, src2 = before[:, :H], before[:, H:H + H2] if H2 else None
            if place == "apart":  # rows apart from one another
                out = torch.full((T, H + 1, D + 8), -3.0, dtype=dtype, device="cuda")[:, :H, 8:]
                out2 = torch.full((T, H2, D), -3.0, dtype=dtype, device="cuda") if H2 else None
            else:
                out, out2 = x, x2
            M.dsv4_rope(M.rope_params(x, out, pos, freqs, x2=x2, out2=out2, rope_first=first, rope_halves=halves,
                                      inverse=inverse, scale=scale))
            for a, y in ((src, out), (src2, out2)):
                if a is None:
                    continue
                want = L.rope(f64(a), np.maximum(pos.cpu().numpy(), 0), hf, first, halves, inverse, scale)
                tol = rope_bound(f64(a), want, first, dim, halves, scale, dtype)
                assert np.all((np.abs(f64(y) - want) <= tol)[live])
                kept = f64(a) if place == "in place" else np.full(a.shape, -3.0)
                np.testing.assert_array_equal(f64(y)[~live], kept[~live])
            if place == "in place":
                np.testing.assert_array_equal(f64(fused[:, H + H2:]), f64(before[:, H + H2:]))
    assert M.dsv4_read_device_flags() == 0


def test_rope_of_special_values(M):
    """Infinities and NaN stay within their pair; dims that are copied keep their bits."""
    x = torch.randn((2, 2, 64), device="cuda")
    x[0, 0, 3], x[1, 1, 20], x[0, 1, 50] = math.nan, math.inf, math.nan
    y = torch.zeros_like(x)
    M.dsv4_rope(M.rope_params(x, y, ints([5, 9]), M.rope_freqs(32)))
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, 2:4] = want[1, 1, 20:22] = True
    want[0, 1, 50] = True
    assert torch.equal(bad, want)


def test_rope_offsets_past_32_bits(M):
    """Rows of a buffer of more than 2^32 elements."""
    rows, width = 70000, 1 << 16
    big = torch.empty((rows, width), dtype=BF16, device="cuda")
    x = big[:, :128].unflatten(1, (2, 64))
    last = torch.randn((3, 2, 64), device="cuda").to(BF16)
    x[-3:] = last
    pos = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    pos[-3:] = ints([4, 99, 100000])
    freqs = M.rope_freqs(64)
    M.dsv4_rope(M.rope_params(x, x, pos, freqs))
    want = L.rope(f64(last), [4, 99, 100000], freqs.cpu().numpy())
    assert np.all(np.abs(f64(x[-3:]) - want) <= rope_bound(f64(last), want, 0, 64, False, 1.0, BF16))


@pytest.mark.parametrize("rows,dim,first,scale", [(1, 8, 0, 1.0), (4097, 64, 0, 1.3), (333, 96, 2 ** 31 - 400, -1.0),
                                                  (70, 1024, 1 << 20, 1.0), (100, 40, 17, 0.5)])
def test_rope_table(M, rows, dim, first, scale):
    freqs = M.rope_freqs(dim, theta=160000.0, scaling="bands", factor=8.0, original_len=8192)
    table = torch.full((rows + 1, dim), 7.0, device="cuda")
    M.dsv4_rope_table(M.rope_table_params(table[:rows], freqs, first_position=first, scale=scale))
    w = L.angles(np.arange(first, first + rows), freqs.cpu().numpy())
    want = scale * np.concatenate([np.cos(w), np.sin(w)], 1)
    # pi 2^-24 of the angle, two steps of the sums, the factor's rounding
    assert np.abs(f64(table[:rows]) - want).max() <= abs(scale) * 7 * 2.0 ** -24
    small = np.abs(np.sin(w)) < 2.0 ** -9  # near 0 the sine is as exact relatively
    err = np.abs(f64(table[:rows])[:, dim // 2:] - want[:, dim // 2:])
    assert np.all(err[small] <= 8 * 2.0 ** -24 * np.abs(want[:, dim // 2:][small]) + 1e-18)
    assert torch.all(table[rows] == 7.0)


def test_rope_agrees_with_the_append_over_its_table(M):
    """Keys that the append turns by dsv4_rope_table's rows and keys that dsv4_rope turns: a rounding of bf16 apart at
    most."""
    from gqa_cases import Batch, dev
    bt = Batch([70, 1, 40], [200, 33, 40], 4, 2, 64, 16, "bf16", seed=5)
    freqs = M.rope_freqs(32, scaling="linear", factor=2.0)
    table = torch.empty((256, 32), device="cuda")
    M.dsv4_rope_table(M.rope_table_params(table, freqs))
    q, k, v = dev(bt.q), dev(bt.k_new), dev(bt.v_new)
    kc, vc = (dev(c) for c in bt.caches)
    q_out = torch.empty_like(q)
    M.dsv4_gqa_append(M.gqa_append_params(k, v, kc, vc, dev(bt.table), dev(bt.q_start), dev(bt.kv), bt.max_q,
                                          cos_sin=table, rope_first=32, rope_halves=True, q=q, q_out=q_out))
    pos = ints(np.concatenate([np.arange(bt.kv[b] - bt.n[b], bt.kv[b]) for b in range(3)]))
    y = torch.empty_like(q)
    M.dsv4_rope(M.rope_params(q, y, pos, freqs, rope_first=32, rope_halves=True))
    a, b = y.double(), q_out.double()
    # (fp32 results 2^-20 of |a| + |b| apart, then one rounding each)
    assert torch.all((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs()) + 2.0 ** -16)


# ------------------------------------------------------------------------------------------------
# batch plan
# ------------------------------------------------------------------------------------------------
class Requests:
    """A batch that has been running: every request holds pages for up to three rows more than it kept."""

    def __init__(self, seed, B, specs, ctx, n_max, free, T=None, width=None, ended=0.1, fresh=0.1):
        g = self.g = np.random.default_rng(seed)
        self.ctx = g.integers(1, ctx + 1, B)
        self.add = g.integers(0, 5, B)
        self.n = g.integers(0, n_max + 1, B)
        new, end = g.random(B) < fresh, g.random(B) < ended
        rows = self.ctx + self.add + g.integers(0, 4, B)
        rows[new] = 0
        self.ctx[new | end], self.add[new | end], self.n[end] = 0, 0, 0
        self.T = int(self.n.sum()) + 5 if T is None else T
        self.caches = []
        for page, ratio, window in specs:
            held = -(-(rows // ratio) // page)
            first = np.minimum(held, np.maximum(0, self.ctx - window + 1) // page) if window else np.zeros(B, np.int64)
            first[new | end] = 0
            need = -(-((self.ctx + self.add + self.n) // ratio) // page)
            w = int(max(held.max(initial=0), need.max(initial=0), 1)) + 2 if width is None else width
            total = int((held - first).sum()) + free
            order = g.permutation(total)
            table = np.full((B, w), -7, np.int64)
            at = 0
            for b in range(B):
                m = held[b] - first[b]
                table[b, first[b]:held[b]] = order[at:at + m]
                at += m
            stack = np.full(total, -9, np.int64)
            stack[:free] = order[at:]
            self.caches.append(L.Cache(page, ratio, window, table, held, first, stack, free))

    def device(self, M, in_place=False, slots=True, outputs=True):
        """The call's parameters and the tensors that it writes."""
        B, T = len(self.ctx), self.T
        new = lambda n, dt=torch.int32: torch.full((n,), -5, dtype=dt, device="cuda")  # noqa: E731
        t = {"ctx": ints(self.ctx), "add": ints(self.add), "n": ints(self.n), "q_start": new(B + 1), "kv_len": new(B),
             "pos": new(T) if outputs else None, "seq": new(T) if outputs else None, "k": []}
        t["ctx_out"] = t["ctx"] if in_place else new(B)
        caches = []
        for c in self.caches:
            d = {"table": ints(c.table), "held": ints(c.held), "first": ints(c.first), "stack": ints(c.stack),
                 "count": ints([c.count]), "slots": new(T, torch.int64) if slots else None}
            for name, size in (("held", B), ("first", B), ("count", 1)):
                d[name + "_out"] = d[name] if in_place else new(size)
            caches.append(M.plan_cache(d["table"], d["held"], d["stack"], d["count"], c.page, held_out=d["held_out"],
                                       free_count_out=d["count_out"], ratio=c.ratio, window=c.window,
                                       first=d["first"] if c.window else None,
                                       first_out=d["first_out"] if c.window else None, slots=d["slots"]))
            t["k"].append(d)
        p = M.batch_plan_params(t["ctx"], t["n"], t["q_start"], t["kv_len"], caches, ctx_add=t["add"],
                                ctx_out=t["ctx_out"], positions=t["pos"], token_seq=t["seq"], max_tokens=T)
        return p, t

    def check(self, t):
        """Compares with the definition (and advances this object's caches)."""
        r = L.plan(self.ctx, self.add, self.n, self.T, self.caches)
        eq = lambda a, b, what: np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=what)  # noqa: E731
        for name in ("ctx_out", "q_start", "kv_len"):
            eq(t[name], r[name], name)
        if t["pos"] is not None:
            eq(t["pos"], r["positions"], "positions")
            eq(t["seq"], r["seq"], "seq")
        for g, (c, d) in enumerate(zip(self.caches, t["k"])):
            eq(d["table"], c.table, f"table {g}")
            eq(d["held_out"], c.held, f"held {g}")
            eq(d["stack"], c.stack, f"stack {g}")
            eq(d["count_out"], [c.count], f"count {g}")
            if c.window:
                eq(d["first_out"], c.first, f"first {g}")
            if d["slots"] is not None:
                eq(d["slots"], r["slots"][g], f"slots {g}")
        return r


PLANS = [  # B, caches (page, ratio, window), ctx, n_max, free pages
    (1, [(64, 1, 0)], 1, 1, 1), (1, [(16, 1, 0)], 100, 5000, 400), (7, [(16, 1, 0)], 60, 4, 9),
    (64, [(64, 1, 128), (64, 4, 0)], 900, 4, 40), (300, [(64, 1, 0)], 3000, 4, 5), (65, [(1, 1, 3)], 20, 6, 600),
    (33, [(128, 1, 500), (256, 4, 0), (64, 128, 0)], 4000, 700, 60), (1000, [(32, 1, 0), (16, 4, 0)], 300, 3, 30),
    (1025, [(16, 1, 40), (8, 3, 0), (64, 128, 0), (5, 7, 0)], 500, 9, 700), (4096, [(64, 1, 0)], 2000, 6, 300),
    (2500, [(16, 1, 0)], 30, 100, 20000), (4096, [(16, 1, 9), (32, 1, 70), (8, 1, 33), (64, 1, 128)], 90, 3, 5000),
    (40, [(64, 1, 0)], 9000, 13000, 9000),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in place"])
@pytest.mark.parametrize("case", PLANS, ids=lambda c: f"B{c[0]}_" + "_".join("-".join(map(str, s)) for s in c[1]) + f"_free{c[4]}")
def test_plan(M, case, in_place):
    B, specs, ctx, n_max, free = case
    q = Requests(B + free, B, specs, ctx, n_max, free)
    p, t = q.device(M, in_place)
    M.dsv4_batch_plan(p)
    assert not q.check(t)["flagged"] and M.dsv4_read_device_flags() == 0


def test_plan_again_is_the_same(M):
    q = Requests(3, 200, [(16, 1, 64), (16, 4, 0)], 700, 5, 100)
    p, t = q.device(M)
    for _ in range(3):
        M.dsv4_batch_plan(p)
    q.check(t)


@pytest.mark.parametrize("T", [0, 1, 63, 200])
def test_plan_with_less_room_than_tokens(M, T):
    q = Requests(4, 100, [(16, 1, 0)], 300, 8, 300, T=T)
    p, t = q.device(M)
    M.dsv4_batch_plan(p)
    r = q.check(t)
    assert r["q_start"][-1] <= T


def test_plan_of_the_largest_step(M):
    """Room for 2^19 tokens, nearly all of them taken."""
    q = Requests(10, 60, [(256, 1, 0)], 2000, 17000, 3000, T=1 << 19, ended=0.0)
    p, t = q.device(M)
    M.dsv4_batch_plan(p)
    assert q.check(t)["q_start"][-1] > 1 << 18


def test_plan_empty_batches(M):
    for B in (0, 5):
        q = Requests(5, B, [(16, 1, 0)], 50, 0 if B else 3, 4, T=9, width=8, ended=0.0, fresh=0.0)
        p, t = q.device(M)
        M.dsv4_batch_plan(p)
        q.check(t)
        assert torch.all(t["pos"] == -1) and torch.all(t["k"][0]["slots"] == -1)


def test_plan_without_optional_outputs(M):
    q = Requests(6, 40, [(16, 1, 0), (16, 4, 0)], 90, 4, 50)
    p, t = q.device(M, slots=False, outputs=False)
    M.dsv4_batch_plan(p)
    q.check(t)


def test_plan_flags_and_leaves_bad_requests(M):
    """Negative and oversized counts, tables too short, held and first out of order, a window before first: those
    requests are left alone and flagged, the others planned."""
    q = Requests(7, 40, [(16, 1, 32), (16, 4, 0)], 400, 4, 200, ended=0.0, fresh=0.0)
    q.ctx[3], q.n[5], q.add[7], q.n[9], q.ctx[11] = -50, -1, -2 ** 31, 2 ** 31 - 1, 2 ** 30
    a, c = q.caches
    a.first[13], a.held[15], c.held[17], c.held[19] = -1, 999, -4, 10 ** 6
    a.first[21] = a.held[21] + 1
    q.ctx[23] = 1
    q.add[23] = 0
    a.first[23] = a.held[23]
    p, t = q.device(M)
    M.dsv4_batch_plan(p)
    r = q.check(t)
    assert r["flagged"] and M.dsv4_read_device_flags() == 1
    assert M.dsv4_read_device_flags() == 0


@pytest.mark.parametrize("count,ended,bad", [(-3, 0.4, True), (10 ** 6, 0.4, True), (None, 0.4, False), (None, 0.0, True)])
def test_plan_flags_bad_stacks(M, count, ended, bad):
    """A count out of range, or one that leaves no room for what is given back; pages out of range on the stack: below
    what is given back, so that none is popped, and on top."""
    q = Requests(8, 30, [(16, 1, 0)], 200, 20, 100, ended=ended)
    c = q.caches[0]
    if count is None:
        c.stack[90:100] = [-1, 10 ** 6] * 5
    else:
        c.count = count
    p, t = q.device(M)
    M.dsv4_batch_plan(p)
    assert q.check(t)["flagged"] == bad and M.dsv4_read_device_flags() == int(bad)


def test_plan_steps_of_a_loop(M):
    """Fifty steps in place over fixed buffers, captured once: requests grow, are cut back, end and begin; at every step no
    page is lost or held twice."""
    B, specs = 48, [(16, 1, 40), (16, 4, 0)]
    q = Requests(9, B, specs, 200, 4, 400, width=40, T=64)
    p, t = q.device(M, in_place=True)
    graph, ready = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=ready):
        M.dsv4_batch_plan(p)
    g = np.random.default_rng(1)
    for _ in range(50):
        graph.replay()
        r = q.check(t)
        for c in q.caches:
            mine = np.concatenate([c.table[b, c.first[b]:c.held[b]] for b in range(B)] + [c.stack[:c.count]])
            assert sorted(mine) == list(range(len(c.stack)))
        ran = np.diff(r["q_start"])
        q.ctx = r["ctx_out"].astype(np.int64)
        q.add = np.where(ran > 0, g.integers(1, 5, B).clip(max=np.maximum(ran, 1)), 0)
        q.n = np.where(q.n == 0, g.integers(1, 30, B), g.integers(1, 5, B))
        end = (g.random(B) < 0.05) | (q.ctx + q.add > 560)
        q.ctx[end], q.add[end], q.n[end] = 0, 0, 0
        for name in ("ctx", "add", "n"):
            t[name].copy_(ints(getattr(q, name)))
    assert M.dsv4_read_device_flags() == 0


# ------------------------------------------------------------------------------------------------
# verification of drafted tokens
# ------------------------------------------------------------------------------------------------
class Drafts:
    def __init__(self, seed, n, V, target=BF16, draft=BF16, target_probs=False, draft_probs=False, greedy=0.0, stride=0,
                 pad=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.target_probs, self.draft_probs, self.V = target_probs, draft_probs, V
        n = np.asarray(n)
        B = len(n)
        self.start = np.concatenate([[0], np.cumsum(n)])
        T = int(self.start[-1]) + pad
        self.T, self.B, self.W = T, B, max(1, int(n.max(initial=0)))
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.temp = 0.5 + torch.rand((B,), generator=g, device="cuda")
        self.temp[torch.rand((B,), generator=g, device="cuda") < greedy] = 0.0
        seq = np.repeat(np.arange(B), n)
        of_row = torch.cat([self.temp[ints(seq, torch.long)], torch.ones(pad, device="cuda")])
        of_row = torch.where(of_row > 0, of_row, 1.0)[:, None]
        z = r(T, V) * spread
        z.scatter_(1, torch.randint(0, V, (T, 6), generator=g, device="cuda"), 6 + 2 * r(T, 6))
        y = z + 0.4 * r(T, V)
        place = lambda x, dt: self._rows(x, dt, stride)  # noqa: E731
        p, q = torch.softmax(z / of_row, 1), torch.softmax(y / of_row, 1)
        self.target = place(p if target_probs else z, target)
        drawn = (q / torch.empty_like(q).exponential_(generator=g)).argmax(1).cpu().numpy()
        best = y.argmax(1).cpu().numpy()
        self.tokens = torch.randint(0, V, (T,), generator=g, device="cuda").cpu().numpy()
        self.draft, rows = None, []
        for b in range(B):
            for t in range(self.start[b], self.start[b + 1] - 1):
                self.tokens[t + 1] = best[t] if self.temp[b] == 0 else drawn[t]
                rows.append(t)
        if draft is not None:
            self.draft = place((q if draft_probs else y)[rows], draft)
        self.u = torch.rand((T,), generator=g, device="cuda")
        self.noise = place(torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_(min=1e-20), F32)
        self.draft_row = None

    @staticmethod
    def _rows(x, dtype, stride):
        """Rows `stride` elements further apart than they are long, from an odd element on."""
        if not stride:
            return x.to(dtype)
        big = torch.full((x.shape[0] * (x.shape[1] + stride) + 1,), math.nan, dtype=dtype, device="cuda")
        view = big[1:].unflatten(0, (x.shape[0], -1))[:, :x.shape[1]] if x.shape[0] else x.to(dtype)
        view.copy_(x)
        return view

    def device(self, M, sampled=True, logp=True, temperature=True):
        t = {"out": torch.full((self.B, self.W), -5, dtype=torch.int32, device="cuda"),
             "count": torch.full((self.B,), -5, dtype=torch.int32, device="cuda"),
             "logp": torch.full((self.B, self.W), -5.0, device="cuda") if logp else None}
        p = M.draft_verify_params(
            self.target, ints(self.tokens), ints(self.start), self.W, t["out"], t["count"], draft=self.draft,
            draft_row=None if self.draft_row is None else ints(self.draft_row),
            temperature=self.temp if temperature else None, u=self.u if sampled else None,
            noise=self.noise if sampled else None, logp=t["logp"], target_probs=self.target_probs,
            draft_probs=self.draft_probs)
        return p, t

    def want(self, sampled=True, temperature=True):
        return L.verify(f64(self.target), self.tokens, self.start, self.W,
                        draft=None if self.draft is None else f64(self.draft), draft_row=self.draft_row,
                        temperature=self.temp.double().cpu().numpy() if temperature else None,
                        u=f64(self.u) if sampled else None, noise=f64(self.noise) if sampled else None,
                        target_probs=self.target_probs, draft_probs=self.draft_probs)

    def run(self, M, flags=0, telling=True, **kw):
        p, t = self.device(M, **kw)
        M.dsv4_draft_verify(p)
        assert M.dsv4_read_device_flags() == flags
        return self.check(t, telling, **kw)

    def check(self, t, telling=True, logp=True, **kw):
        out, count, lp, margin = self.want(**kw)
        got, n = t["out"].cpu().numpy(), t["count"].cpu().numpy()
        # A weight's relative error: its exponent's argument (2^-23 of up to 2^7, carried along to 2^-30), the special
        # function (2^-22) and a few roundings; a row's sum adds the terms' errors and vocab / 2^9 additions.
        rel = 2.0 ** -20 + (self.V / 512 + 32) * 2.0 ** -24
        for b in range(self.B):
            same = n[b] == count[b] and np.array_equal(got[b], out[b])
            assert same or margin[b] < 4 * rel, (b, n[b], count[b], got[b], out[b], margin[b])
            if same and logp:
                live = out[b] >= 0
                tol = rel + 2.0 ** -22 * np.abs(lp[b][live]) + 13 * 2.0 ** -23
                assert np.all(np.abs(f64(t["logp"][b])[live] - lp[b][live]) <= tol)
                assert torch.all(t["logp"][b].cpu()[torch.from_numpy(~live)] == 0)
        # few decisions are open, so that the check above means something (low temperatures put p and q within
        # 2^-24 of 1, and their difference with them)
        assert not telling or (margin < 4 * rel).sum() <= max(1, self.B // 50)
        return out, count


KINDS = [(BF16, BF16, False, False), (F32, F32, False, True), (BF16, F32, True, True), (F32, None, False, False),
         (F32, BF16, True, False), (BF16, None, True, False), (F32, F32, False, False), (BF16, F32, False, True)]
SIZES = [(1, [1]), (1, [3, 1]), (2, [4, 2, 1]), (7, [1, 5]), (33, [4] * 9), (1000, [3, 0, 1, 8, 2]), (4099, [4] * 20),
         (32000, [4, 4]), (8192, [1] * 40), (20011, [9, 17, 1]), (129, [2] * 700)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "_".join("none" if x is None else str(x).replace("torch.", "") for x in k))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"V{s[0]}_B{len(s[1])}_n{max(s[1])}")
def test_verify(M, size, kind):
    V, n = size
    Drafts(V + len(n), n, V, *kind, greedy=0.2).run(M)


@pytest.mark.parametrize("stride", [1, 3, 8, 37])
@pytest.mark.parametrize("kind", KINDS[:3], ids=["bf16", "fp32", "probs"])
def test_verify_rows_of_any_alignment(M, kind, stride):
    Drafts(stride, [4, 3, 5], 3001, *kind, stride=stride, greedy=0.3).run(M)


def test_verify_large_vocabulary(M):
    Drafts(11, [4, 2], 1 << 18, F32, BF16).run(M)
    Drafts(12, [3], 151936, BF16, None, greedy=0.0).run(M)


def test_verify_padding_behind_the_batch(M):
    d = Drafts(13, [3, 2], 500, pad=7)
    d.target[5:] = math.nan
    d.run(M)


def test_verify_all_greedy_forms(M):
    """Without u and noise every sequence is greedy, whatever its temperature; without temperatures none is."""
    d = Drafts(14, [4] * 12, 700, draft=None)
    d.run(M, sampled=False)
    d.run(M, sampled=False, temperature=False)
    d.run(M, temperature=False)
    d.run(M, logp=False)


def test_verify_greedy_ties_go_to_the_first(M):
    """The maximum at several places, within one thread's elements, across warps and CTAs: the lowest index."""
    V = 50000
    for places in ([3, 4], [3, 49999], [8, 16, 24], [24999, 25000, 7], [12345, 31, 40000]):
        d = Drafts(15, [2], V, BF16, None, greedy=1.1)
        d.target[:, places] = 40.0
        d.tokens[1] = max(places)          # (a maximum, but not the first)
        out, count = d.run(M)
        assert count[0] == 1 and out[0, 0] == min(places)
        d.tokens[1] = min(places)
        assert d.run(M)[1][0] == 2


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_verify_masks_and_special_values(M, dtype):
    """Masked by -inf, by the type's lowest value and by NaN; rows with nothing left; a lone +inf."""
    lowest = torch.finfo(dtype).min
    d = Drafts(16, [4] * 8, 300, dtype, dtype)
    d.target[:, ::2] = -math.inf
    d.target[0:4, 1:200:2] = lowest
    d.target[4:8, 1:100:2] = math.nan
    d.target[8] = -math.inf                # nothing is left in the first row of sequence 2
    d.target[13] = math.nan                # and in the second of sequence 3
    d.target[16, 17] = math.inf
    d.tokens[13] = 5                       # (whatever the draft: sequence 3's first row decides)
    d.draft[6] = -math.inf                 # nothing left in a draft row: q = 0
    d.draft[9, :150] = math.nan
    out, count = d.run(M)
    assert count[2] == 0 and out[2, 0] == -1
    lone = Drafts(17, [1], 300, dtype, None)
    lone.target[0] = -math.inf
    lone.target[0, 299] = lowest
    out, count = lone.run(M)
    assert out[0, 0] == 299 and count[0] == 1


def test_verify_probabilities_of_special_values(M):
    d = Drafts(18, [3] * 6, 200, F32, F32, True, True)
    d.target[0, :100] = math.nan
    d.target[3, :100] = -1.0
    d.target[6] = 0.0
    d.draft[2, :] = math.nan
    out, count = d.run(M)
    assert count[2] == 0 and out[2, 0] == -1


def test_verify_where_nothing_is_left_of_the_difference(M):
    """p <= q everywhere (sums below 1 are allowed): the race runs over p."""
    d = Drafts(19, [2] * 5, 400, F32, F32, True, True)
    d.draft.copy_(d.target[0::2] * 3)
    d.u.fill_(0.9999)
    d.run(M)


def test_verify_identical_models_keep_every_draft(M):
    d = Drafts(20, [5] * 10, 1000, F32, F32)
    for b in range(10):
        for i in range(4):
            d.draft[4 * b + i] = d.target[5 * b + i]
    d.u.clamp_(max=0.999)
    _, count = d.run(M)
    assert np.all(count == 5)


@pytest.mark.parametrize("temp", [1e-38, 1e-6, 0.01, 100.0, 1e38, math.inf, -1.0, math.nan])
def test_verify_temperatures(M, temp):
    """Down to where only the maximum is left, up to where every token is as likely; not over 0: greedy."""
    d = Drafts(21, [3] * 6, 600, F32, F32)
    d.temp.fill_(temp)
    d.run(M, telling=not 0 < temp < 0.1)


def test_verify_draft_rows_in_any_order(M):
    """draft_row names each drafted token's row, the same row for several."""
    d = Drafts(22, [4] * 6, 900)
    perm = np.random.default_rng(2).permutation(len(d.draft))
    row = np.full(d.T, -3)
    at = 0
    for b in range(6):
        for t in range(d.start[b], d.start[b + 1] - 1):
            row[t + 1] = perm[at]
            at += 1
    shuffled = torch.empty_like(d.draft)
    shuffled[ints(perm, torch.long)] = d.draft
    d.draft, d.draft_row = shuffled, row
    d.run(M)
    d.draft_row = np.where(row >= 0, 3, row)
    d.run(M)


def test_verify_flags_tokens_and_rows_out_of_range(M):
    d = Drafts(23, [4] * 5, 300)
    d.tokens[[1, 6]] = [-1, 300]
    d.run(M, flags=1)
    d = Drafts(24, [4] * 5, 300)
    d.draft_row = np.arange(d.T) - np.repeat(np.arange(5), 4) - 1
    d.draft_row[[1, 7]] = [-1, 10 ** 6]
    d.run(M, flags=1)
    d = Drafts(25, [4] * 5, 300, draft=None)
    d.tokens[[1, 6]] = [-2 ** 31, 2 ** 31 - 1]
    d.run(M, flags=1)


@pytest.mark.parametrize("start", [[0, 3, 2, 9], [0, -1, 5, 9], [0, 3, 8, 9], [0, 3, 12, 9]])
def test_verify_skips_bad_sequences(M, start):
    """q_start out of order, below 0, longer than the bound or past T: skipped, their outputs stay, and flagged."""
    d = Drafts(26, [3, 3, 3], 300)
    p, t = d.device(M)
    bad = ints(start)
    p.q_start, keep = bad.data_ptr(), bad
    M.dsv4_draft_verify(p)
    assert M.dsv4_read_device_flags() == 1
    for b in range(3):
        if not 0 <= start[b] <= start[b + 1] <= 9 or start[b + 1] - start[b] > 3:
            assert torch.all(t["out"][b] == -5) and t["count"][b] == -5 and torch.all(t["logp"][b] == -5)
    del keep


def test_verify_offsets_past_32_bits(M):
    """Target, draft and noise rows behind 2^32 elements."""
    V, n = 1000, 3
    d = Drafts(27, [n], V, BF16, BF16)
    stride = (1 << 31) + 8
    far = lambda x: torch.empty((x.shape[0] - 1) * stride + V, dtype=x.dtype, device="cuda").as_strided(x.shape, (stride, 1))  # noqa: E731
    for name in ("target", "draft"):
        big = far(getattr(d, name))
        big.copy_(getattr(d, name))
        setattr(d, name, big)
    d.run(M)


@pytest.mark.parametrize("shift", [-1e7, -3000.0, 3000.0, 1e7, 1e30])
@pytest.mark.parametrize("V", [100, 40000])
def test_verify_logits_far_from_zero(M, shift, V):
    """Exponents beyond the range of the quick sums, and rows that lie there altogether."""
    d = Drafts(30, [3] * 6, V, F32, F32, greedy=0.2)
    d.target += shift
    d.draft -= shift
    d.run(M, telling=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("order", ["up", "down", "late", "jumps"])
def test_verify_logits_that_rise_along_the_row(M, dtype, order):
    """The reference of the sums is found at the row's begin and has to follow what comes later."""
    V = 30000
    d = Drafts(31, [3] * 6, V, dtype, dtype, greedy=0.2)
    at = torch.arange(V, device="cuda").float() / V
    slope = {"up": 150 * at, "down": -150 * at, "late": torch.where(at > 0.999, 300.0, 0.0),
             "jumps": 60 * torch.floor(at * 7)}[order]
    d.target.copy_((d.target.float() + slope).to(dtype))
    d.draft.copy_((d.draft.float() + slope).to(dtype))
    d.run(M, telling=False)


def test_verify_masked_stretches(M):
    """Most of the vocabulary masked, by -inf and by the lowest value: slices of CTAs and warps with nothing left."""
    for dtype in (BF16, F32):
        for mask in (-math.inf, torch.finfo(dtype).min):
            for keep in (slice(0, 7), slice(29990, 30000), slice(15000, 15003), slice(8, 29992, 4000)):
                d = Drafts(32, [3] * 4, 30000, dtype, dtype, greedy=0.3)
                kept = d.target[:, keep].clone()
                d.target.fill_(mask)
                d.target[:, keep] = kept
                d.run(M, telling=False)


def test_verify_ties_of_the_race_go_to_the_first(M):
    """Equal probabilities over equal noise: the lowest index, wherever the others are."""
    V = 60000
    d = Drafts(33, [1] * 4, V, F32, None)
    d.target.fill_(-5.0)
    d.noise.fill_(1.0)
    for b, places in enumerate(([5, 6], [59999, 31], [30000, 29999, 15000], [7500, 52499, 8])):
        d.target[b, places] = 2.0
    out, count = d.run(M, telling=False)
    assert list(out[:, 0]) == [5, 31, 15000, 8]


def test_verify_empty_inputs(M):
    """No tokens at all, and drafted tokens whose draft has no row."""
    d = Drafts(34, [0, 0, 0], 100)
    p, t = d.device(M)
    M.dsv4_draft_verify(p)
    assert torch.all(t["count"] == 0) and torch.all(t["out"] == -1) and M.dsv4_read_device_flags() == 0
    d = Drafts(35, [2, 2], 100)
    d.draft = d.draft[:0]
    out, count = d.run(M, flags=1)
    assert np.all(count == 1)


def test_verify_a_million_logits(M):
    Drafts(36, [3, 1], 1 << 20, BF16, BF16, stride=5).run(M)


def test_two_streams_at_once(M):
    """Calls of each kind side by side on two streams, each over its own buffers."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    ds = [Drafts(40 + i, [4] * 10, 20000) for i in range(2)]
    qs = [Requests(50 + i, 100, [(16, 1, 0), (16, 4, 0)], 300, 4, 200) for i in range(2)]
    vs, ps = [d.device(M) for d in ds], [q.device(M) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            M.dsv4_draft_verify(vs[i][0], stream=s)
            M.dsv4_batch_plan(ps[i][0], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        ds[i].check(vs[i][1])
        qs[i].check(ps[i][1])


def test_rope_reads_broadcast_rows(M):
    """One row for every head, and one token's rows for every token."""
    x = torch.randn((5, 1, 64), device="cuda")
    pos = ints([0, 3, 9, 100, 7])
    freqs = M.rope_freqs(64)
    for src in (x.expand(5, 6, 64), x[:1].expand(5, 1, 64)):
        y = torch.empty(src.shape, device="cuda")
        M.dsv4_rope(M.rope_params(src, y, pos, freqs))
        want = L.rope(f64(src), pos.cpu().numpy(), freqs.cpu().numpy())
        assert np.all(np.abs(f64(y) - want) <= rope_bound(f64(src), want, 0, 64, False, 1.0, F32))


def test_verify_many_sequences(M):
    Drafts(28, [2, 1, 3, 0] * 2000, 64).run(M)


def test_verify_is_deterministic_and_captured(M):
    """The same bits on every run, on another stream, and from a graph whose inputs change between replays."""
    d = Drafts(29, [4] * 20, 30000, greedy=0.2)
    p, t = d.device(M)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.dsv4_draft_verify(p, stream=side)
    side.synchronize()
    first = {k: v.clone() for k, v in t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.dsv4_draft_verify(p)
    for _ in range(5):
        for v in t.values():
            v.fill_(-5)
        graph.replay()
        assert all(torch.equal(t[k], first[k]) for k in t)
    d.check(t)
    d.u.copy_(torch.rand_like(d.u))
    d.noise.copy_(d.noise.flip(1))
    graph.replay()
    d.check(t)


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
def test_decode_loop(M):
    """Steps of a drafted decode over one captured graph: plan -> append and attention of a grouped-query layer -> logits
    -> verification, whose count advances the plan of the next step; every step against the definitions, and the
    attention against one over the rows that should be there."""
    B, k, H, Hkv, D, page, V, width = 6, 3, 4, 2, 64, 16, 512, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    T = B * (k + 1)
    new = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    pages = B * width
    freqs = M.rope_freqs(D)
    cos_sin = torch.empty((width * page, D), device="cuda")
    M.dsv4_rope_table(M.rope_table_params(cos_sin, freqs))
    ctx, add, n = new(B), new(B), torch.full((B,), k + 1, dtype=torch.int32, device="cuda")
    q_start, kv_len, pos = new(B + 1), new(B), new(T)
    table, held, slots = new(B, width), new(B), new(T, dt=torch.int64)
    stack, count = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.tensor([pages], dtype=torch.int32, device="cuda")
    plan = M.batch_plan_params(ctx, n, q_start, kv_len, [M.plan_cache(table, held, stack, count, page, slots=slots)],
                               ctx_add=add, ctx_out=ctx, positions=pos)
    kc, vc = (torch.zeros((pages, Hkv, page, D), dtype=BF16, device="cuda") for _ in range(2))
    qkv = new(T, H + 2 * Hkv, D, dt=BF16)
    q, kn, vn = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    q_rot, out = new(T, H, D, dt=BF16), new(T, H, D, dt=F32)
    append = M.gqa_append_params(kn, vn, kc, vc, table, q_start, kv_len, k + 1, cos_sin=cos_sin, q=q, q_out=q_rot)
    attend = M.gqa_attention_params(q_rot, kc, vc, table, q_start, kv_len, k + 1, width * page, D ** -0.5, out)
    M.gqa_set_workspace(attend, torch.empty(M.dsv4_gqa_attention_workspace_bytes(attend), dtype=torch.uint8, device="cuda"))
    head = r(H * D, V) / 4
    logits, draft = torch.empty((T, V), device="cuda"), torch.empty((B * k, V), device="cuda")
    tokens, u, noise = new(T), torch.empty(T, device="cuda"), torch.empty((B, V), device="cuda")
    words = new(B, k + 1)
    verify = M.draft_verify_params(logits, tokens, q_start, k + 1, words, add, draft=draft, u=u, noise=noise)

    def step():
        M.dsv4_batch_plan(plan)
        M.dsv4_gqa_append(append)
        M.dsv4_gqa_attention(attend)
        torch.matmul(out.view(T, -1), head, out=logits)
        M.dsv4_draft_verify(verify)

    step()                                # (the library product's warm-up)
    for t in (ctx, add, held):
        t.zero_()
    stack.copy_(torch.arange(pages))
    count.fill_(pages)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rows = [[] for _ in range(B)]         # (k, v) of every row that stands, float64
    kept = np.zeros(B, int)
    for _ in range(12):
        qkv.copy_(r(T, H + 2 * Hkv, D))
        draft.copy_(r(B * k, V) * 2)
        tokens.copy_(torch.randint(0, V, (T,), generator=g, device="cuda"))
        u.copy_(torch.rand(T, generator=g, device="cuda") * 0.05)   # (small: some drafts stand)
        noise.exponential_(generator=g)
        before = add.cpu().numpy().copy()
        graph.replay()
        kept = kept + before
        np.testing.assert_array_equal(ctx.cpu().numpy(), kept)
        np.testing.assert_array_equal(kv_len.cpu().numpy(), kept + k + 1)
        np.testing.assert_array_equal(pos.cpu().numpy().reshape(B, -1), kept[:, None] + np.arange(k + 1))
        want, cnt, _, margin = L.verify(f64(logits), tokens.cpu().numpy(), q_start.cpu().numpy(), k + 1, draft=f64(draft),
                                        u=f64(u), noise=f64(noise))
        if margin.min() > 2 ** -16:
            np.testing.assert_array_equal(words.cpu().numpy(), want)
            np.testing.assert_array_equal(add.cpu().numpy(), cnt)
        turned = L.rope(f64(kn), pos.cpu().numpy(), freqs.cpu().numpy())
        qt = f64(q_rot)
        got = f64(out)
        for b in range(B):
            del rows[b][kept[b]:]
            rows[b] += [(turned[b * (k + 1) + i], f64(vn)[b * (k + 1) + i]) for i in range(k + 1)]
            for i in range(k + 1):
                t = b * (k + 1) + i
                for h in range(H):
                    ks = np.stack([x[0][h // (H // Hkv)] for x in rows[b][:kept[b] + i + 1]])
                    vs = np.stack([x[1][h // (H // Hkv)] for x in rows[b][:kept[b] + i + 1]])
                    z = ks @ qt[t, h] * D ** -0.5
                    w = np.exp(z - z.max())
                    # keys are stored as bf16 (2^-8 of each: sum |q k| up to about 100, times 1/8), weights rounded likewise
                    assert np.abs(w @ vs / w.sum() - got[t, h]).max() < 0.25
    assert M.dsv4_read_device_flags() == 0
    assert int(count) + int(held.sum()) == pages
