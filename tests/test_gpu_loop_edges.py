"""The calls around the layers where they can go wrong: what the tests beside their definitions pass over."""
import numpy as np
import pytest
import torch

from oracle import loop_oracle as L
from test_gpu_loop import BF16, F32, Drafts, M, Requests, f64, ints  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------
# draft rows behind sequences without tokens
# ------------------------------------------------------------------------------------------------
def rows_in_order(n):
    """The draft row of every token, counted token by token (-3: not drafted)."""
    row, at = [], 0
    for k in n:
        for i in range(k):
            row.append(-3 if i == 0 else at)
            at += i > 0
    return np.array(row, np.int64)


EMPTIES = [[0, 2], [0, 0, 2], [2, 0, 2], [4, 0, 4], [0, 3, 0, 0, 1, 5, 0, 2, 0], [1, 0, 1, 0, 3],
           np.random.default_rng(0).integers(0, 4, 700).tolist(), [0] * 300 + [3] * 5 + [0] * 2100 + [2, 4]]


@pytest.mark.parametrize("draft,draft_probs", [(BF16, False), (F32, True)], ids=["logits", "probs"])
@pytest.mark.parametrize("n", EMPTIES, ids=lambda n: f"B{len(n)}_first{n[0]}_T{sum(n)}")
def test_verify_draft_rows_behind_empty_sequences(M, n, draft, draft_probs):  # noqa: F811
    """Drafts in order give what the same rows give by name."""
    d = Drafts(len(n) + sum(n), n, 257, F32, draft, draft_probs=draft_probs)
    row = rows_in_order(n)
    assert row.max() + 1 == len(d.draft)
    d.draft_row = row
    named, t = d.device(M)
    M.dsv4_draft_verify(named)
    want = {k: v.clone() for k, v in t.items()}
    d.check(t, telling=len(n) > 20)
    d.draft_row = None
    in_order, t = d.device(M)
    M.dsv4_draft_verify(in_order)
    assert M.dsv4_read_device_flags() == 0
    for k in t:
        assert torch.equal(t[k], want[k]), k


def test_drafted_loop_with_requests_left_out(M):  # noqa: F811
    """Plan and verification of one captured step: requests end, begin and are left out for want of pages, so that sequences
    without tokens lie between the others; the drafts' rows follow one another."""
    B, k, V, page = 24, 3, 300, 4
    W = k + 1
    q = Requests(3, B, [(page, 1, 0)], 20, W, 12, width=20, T=B * W)
    p, t = q.device(M, in_place=True)
    g = torch.Generator(device="cuda").manual_seed(8)
    rng = np.random.default_rng(8)
    target = torch.zeros((q.T, V), device="cuda")
    draft = torch.zeros((q.T, V), device="cuda")
    tokens, u, noise = torch.zeros(q.T, dtype=torch.int32, device="cuda"), torch.zeros(q.T, device="cuda"), torch.ones((B, V), device="cuda")
    words = torch.zeros((B, W), dtype=torch.int32, device="cuda")
    v = M.draft_verify_params(target, tokens, t["q_start"], W, words, t["add"], draft=draft, u=u, noise=noise)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.dsv4_batch_plan(p)
        M.dsv4_draft_verify(v)
    between = 0
    for step in range(25):
        target.normal_(generator=g).mul_(2)
        draft.copy_(target.roll(1, 1) + 0.1)
        noise.exponential_(generator=g).clamp_(min=1e-20)
        u.uniform_(generator=g).mul_(0.2)
        graph.replay()
        r = q.check(t)
        n = np.diff(r["q_start"])
        between += int(np.any((n == 0)[:np.max(np.nonzero(n)[0], initial=0)]))
        row = np.full(q.T, -3)
        known = rows_in_order(n)
        row[:len(known)] = known
        out, count, _, margin = L.verify(f64(target), tokens.cpu().numpy(), r["q_start"], W, draft=f64(draft), draft_row=row,
                                         u=f64(u), noise=f64(noise))
        sure = margin > 2.0 ** -17
        np.testing.assert_array_equal(words.cpu().numpy()[sure], out[sure])
        np.testing.assert_array_equal(t["add"].cpu().numpy()[sure], count[sure])
        q.ctx = r["ctx_out"].astype(np.int64)
        q.add = t["add"].cpu().numpy().astype(np.int64)
        q.n = np.where(q.n == 0, rng.integers(1, W + 1, B), rng.integers(1, W + 1, B))
        end = (rng.random(B) < 0.15) | (q.ctx + q.add > 60)
        q.ctx[end], q.add[end], q.n[end] = 0, 0, 0
        for name in ("ctx", "add", "n"):
            t[name].copy_(ints(getattr(q, name)))
        # the next step's tokens, drawn from the rows that will be theirs
        tokens.copy_(torch.randint(0, V, (q.T,), generator=g, device="cuda"))
    assert between > 10 and M.dsv4_read_device_flags() == 0


# ------------------------------------------------------------------------------------------------
# drafted tokens far below the maximum of their draft row
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("temp", [1e-7, 0.4, 0.5, 1.0, 1.4, 2.0, 100.0])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_verify_drafted_tokens_masked_in_the_draft(M, dtype, temp):  # noqa: F811
    """A drafted token that is the target's maximum stands, however little the draft gave it: u q(x) < p(x) with q(x) next to
    nothing.  (u is below 0.9 and p over 0.99 of what it could be.)"""
    values = [-1e3, -1e6, -1e7, -3e7, -1e8, -1e9, -1e20, -1e30, torch.finfo(dtype).min]
    d = Drafts(70, [2] * len(values), 300, dtype, dtype, spread=0.01 if temp > 10 else 2.0)
    x = torch.arange(len(values), device="cuda") * 31 + 5
    rows = torch.arange(len(values), device="cuda")
    d.tokens[1::2] = x.cpu().numpy()
    d.target[2 * rows, x] = 40.0 if temp < 10 else 3000.0
    d.draft[rows, x] = torch.tensor(values, device="cuda").to(dtype)
    d.temp.fill_(temp)
    d.u.mul_(0.9)
    out, count = d.run(M, telling=False)
    assert np.all(count == 2)


@pytest.mark.parametrize("low", [-1e6, -1e8, -1e30, None])
def test_verify_drafted_tokens_masked_in_the_target(M, low):  # noqa: F811
    """The other way round they fall: p(x) is next to nothing, q(x) is not."""
    d = Drafts(71, [2] * 8, 300, F32, F32)
    rows = torch.arange(8, device="cuda")
    x = torch.from_numpy(d.tokens[1::2].copy()).cuda()
    d.target[2 * rows, x] = torch.finfo(F32).min if low is None else low
    d.u.clamp_(min=1e-3)
    _, count = d.run(M, telling=False)
    assert np.all(count == 1)


def test_verify_drafted_tokens_far_down_in_both(M):  # noqa: F811
    """Both probabilities are too small for a float, their quotient is not: equal rows keep every draft (u below 1)."""
    d = Drafts(72, [2] * 6, 300, F32, F32)
    x = torch.from_numpy(d.tokens[1::2].copy()).cuda()
    rows = torch.arange(6, device="cuda")
    d.draft.copy_(d.target[0::2])
    for row, value in enumerate((-200.0, -1e4, -1e7, -1e9, -1e30, torch.finfo(F32).min)):
        d.target[2 * row, x[row]] = d.draft[row, x[row]] = value
    d.temp.fill_(0.7)
    d.u.clamp_(max=0.999)
    p, t = d.device(M)
    M.dsv4_draft_verify(p)
    d.check(t, telling=False)
    # (beside 1e30 a float64 sum of logarithms loses log u: the definition's count says nothing there)
    assert torch.all(t["count"] == 2) and M.dsv4_read_device_flags() == 0


# ------------------------------------------------------------------------------------------------
# requests without new tokens that hold too few pages
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("free", [1000, 3])
def test_plan_requests_without_tokens_take_nothing(M, free):  # noqa: F811
    """A request that brings no token takes no page and counts for nothing in the admission of those behind it, even where
    it holds fewer pages than its rows need."""
    q = Requests(60, 30, [(16, 1, 0), (8, 4, 0)], 500, 3, free, ended=0.0, fresh=0.0)
    q.n[::3] = 0
    q.T = int(q.n.sum()) + 5
    for c in q.caches:
        c.held[::3] = np.minimum(c.held[::3], 1)
    held = [c.held.copy() for c in q.caches]
    tables = [c.table.copy() for c in q.caches]
    p, t = q.device(M)
    M.dsv4_batch_plan(p)
    q.check(t)
    for i, d in enumerate(t["k"]):
        np.testing.assert_array_equal(d["held_out"].cpu().numpy()[::3], held[i][::3])
        np.testing.assert_array_equal(d["table"].cpu().numpy()[::3], tables[i][::3])
    assert M.dsv4_read_device_flags() == 0


# ------------------------------------------------------------------------------------------------
# log-probabilities next to 0
# ------------------------------------------------------------------------------------------------
def near_one(V, dtype, left, places, temp, stride=0, seed=80):
    """Two sequences a case: a drafted token that is nearly certain, then a last row with a nearly certain token; `left` is
    the probability of all others."""
    n = [2] * len(places)
    d = Drafts(seed, n, V, dtype, dtype, stride=stride)
    d.temp.fill_(temp)
    for b, x in enumerate(places):
        for t, y in ((2 * b, x), (2 * b + 1, V - 1 - x)):
            row = d.target[t].double() / temp
            row[y] = -float("inf")
            others = float(torch.logsumexp(row, 0))
            top = (others + np.log((1 - left) / left)) * temp
            d.target[t, y] = float(top)
        d.tokens[2 * b + 1] = x
        d.draft[b, x] = d.target[2 * b, x]
    d.u.mul_(0.4)
    return d


@pytest.mark.parametrize("greedy", [False, True], ids=["drawn", "greedy"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("left", [0.3, 0.02, 1e-3, 1e-5, 1e-8])
@pytest.mark.parametrize("V,stride", [(40, 0), (2000, 3), (32000, 0), (100003, 1)])
def test_verify_log_probabilities_near_0(M, V, stride, left, dtype, greedy):  # noqa: F811
    """log p = -log(1 + rest / w) is as exact relatively as the other weights' sum.  Of each of these the exponent's
    argument y is off by |y| 2^-22 (a difference, a factor and its own rounding), the special function by 2^-22; V / 512
    additions a lane and 32 after them, the division and the logarithm round once or twice each."""
    places = [0, 1, V - 1, V - 2, V // 2, 7, 8, V // 3]
    d = near_one(V, dtype, left, places, 1.0 if greedy else 0.8, stride)
    if greedy:
        d.temp.fill_(0.0)
    p, t = d.device(M)
    M.dsv4_draft_verify(p)
    out, count, lp, _ = d.want()
    got = f64(t["logp"])
    rows = f64(d.target)
    sure = 0
    for b in range(d.B):
        if count[b] != 2 or int(t["count"][b]) != 2:
            continue
        np.testing.assert_array_equal(t["out"][b].cpu().numpy(), out[b])
        for i in range(2):
            if lp[b, i] < -0.69:
                continue
            z = rows[2 * b + i]
            orders = (z.max() - z.min()) / (1.0 if greedy else 0.8) / np.log(2)
            rel = 2.0 ** -20 + orders * np.log(2) * 2.0 ** -22 + (V / 512 + 40) * 2.0 ** -24
            assert abs(got[b, i] - lp[b, i]) <= rel * abs(lp[b, i]), (b, i, got[b, i], lp[b, i])
            sure += 1
    assert sure >= (0 if left == 0.3 and dtype == BF16 else d.B)


# ------------------------------------------------------------------------------------------------
# offsets past 32 bits, and the plan under the layers that its ratios and windows are for
# ------------------------------------------------------------------------------------------------
def test_verify_every_operand_past_32_bits(M):  # noqa: F811
    """Target, draft and noise rows that decide lie behind 2^32 elements each: indices wrapped to 32 bits, signed or
    not, would read the rows of the others."""
    V = 1000
    d = Drafts(90, [3, 3, 3], V, BF16, BF16)
    for name, stride in (("target", (1 << 29) + 8), ("draft", (1 << 30) - 8), ("noise", (1 << 31) + 4)):
        x = getattr(d, name)
        big = torch.empty((x.shape[0] - 1) * stride + V, dtype=x.dtype, device="cuda").as_strided(x.shape, (stride, 1))
        big.copy_(x)
        setattr(d, name, big)
        assert (x.shape[0] - 1) * stride > 1 << 32
    d.u.mul_(0.5)
    _, count = d.run(M)
    assert count[2] >= 2  # (the last sequence comes to its second draft, whose row is the last)


@pytest.mark.parametrize("ratio,coff", [(4, 2), (128, 1)], ids=["ratio4", "ratio128"])
def test_plan_under_the_compressed_layers(M, ratio, coff):  # noqa: F811
    """Tables and slots of a windowed and a compressed cache under the layers that read them: the insert by slot, the
    compressor, the attention over window and entries.  Beside the same calls over tables that give every sequence pages of
    its own, where nothing is ever given back: rows that are seen, entries and outputs are the same bits, over a captured
    step whose drafts are cut back, with a pool that just holds what the window needs and a request that makes place for another."""
    B, n, page, window, steps, H = 3, 4, 64, 128, 110, 2
    most, width = steps * n + n, steps * n // page + 2
    T = B * n
    g = torch.Generator(device="cuda").manual_seed(ratio)
    rng = np.random.default_rng(ratio)
    new = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    cos_sin = torch.empty((most + 1, 64), device="cuda")
    M.dsv4_rope_table(M.rope_table_params(cos_sin, M.rope_freqs(64)))
    ctx, add, count = new(B), new(B), torch.full((B,), n, dtype=torch.int32, device="cuda")
    q_start, kv_len, pos = new(B + 1), new(B), new(T)
    caches, sides = [], []
    for r, w, pages in ((1, window, 4 * B), (ratio, 0, B * (most // ratio // page + 1))):
        k = {"table": torch.full((B, width), -1, dtype=torch.int32, device="cuda"), "held": new(B), "first": new(B), "pages": pages,
             "stack": torch.randperm(pages, generator=g, device="cuda").int(), "count": torch.tensor([pages], dtype=torch.int32, device="cuda"),
             "slots": new(T, dt=torch.int64)}
        caches.append(M.plan_cache(k["table"], k["held"], k["stack"], k["count"], page, ratio=r, window=w, slots=k["slots"],
                                   first=k["first"] if w else None))
        sides.append(k)
    plan = M.batch_plan_params(ctx, count, q_start, kv_len, caches, ctx_add=add, ctx_out=ctx, positions=pos)
    kv = new(T, 576, dt=BF16)
    score, q = torch.empty((T, 2 * coff * 576), device="cuda"), new(T, H, 576, dt=BF16)
    weight = torch.ones(576, device="cuda")

    class Layer:
        def __init__(self, tables, slots, pages):
            self.tables, self.slots = tables, slots
            self.swa, self.main = (torch.full((p, page, 576), float("nan"), dtype=BF16, device="cuda") for p in pages)
            self.state = torch.zeros((B, coff * ratio, 2 * coff * 576), device="cuda")
            self.out, self.lse = torch.zeros((T, H, 512), device="cuda"), torch.zeros((T, H), device="cuda")
            self.p = M.sparse_mla_params(q, M.BF16, pos, n, self.swa, tables[0], self.main, tables[1], M.BF16, page, ratio, window,
                                         None, None, 576 ** -0.5, self.out, M.F32, self.lse, most)
            self.ws = torch.empty(max(256, M.dsv4_sparse_mla_decode_workspace_bytes(self.p)), dtype=torch.uint8, device="cuda")
            self.p.workspace, self.p.workspace_bytes = self.ws.data_ptr(), self.ws.numel()

        def run(self):
            M.dsv4_kv_insert(kv, M.BF16, self.slots, self.swa, M.BF16, page, positions=pos, cos_sin=cos_sin)
            M.dsv4_compress_update(score, pos, n, ratio, coff, self.state, None, weight, 1e-6, cos_sin, self.main, M.BF16,
                                   self.tables[1], page)
            M.dsv4_sparse_mla_decode(self.p)

    planned = Layer([k["table"] for k in sides], sides[0]["slots"], [k["pages"] for k in sides])
    own = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    plain = Layer([own, own], new(T, dt=torch.int64), [B * width] * 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.dsv4_batch_plan(plan)
        planned.run()
    kept, given = np.zeros(B, int), 0
    for step in range(steps):
        if step == steps // 2:  # sequence 1 ends; another takes its place
            ctx[1], add[1], before = 0, 0, count.clone()
            ctx.add_(add), add.zero_(), count.zero_()
            M.dsv4_batch_plan(plan)
            assert int(kv_len[1]) == 0 and int(sides[0]["held"][1]) == 0
            count.copy_(before)
            kept = ctx.cpu().numpy().astype(int)
            for layer in (planned, plain):
                layer.state[1] = 0
        else:
            kept = kept + add.cpu().numpy()
        kv.normal_(generator=g), score.normal_(generator=g), q.normal_(generator=g)
        graph.replay()
        at = kept[:, None] + np.arange(n)
        np.testing.assert_array_equal(pos.cpu().numpy().reshape(B, n), at)
        plain.slots.copy_(ints((np.arange(B)[:, None] * width * page + at).ravel(), torch.int64))
        plain.run()
        tables = [k["table"].cpu().numpy() for k in sides]
        for b in range(B):
            seen = np.arange(max(0, kept[b] - window + 1), kept[b] + n)
            entries = np.arange((kept[b] + n) // ratio)
            for rows, table, mine, theirs in ((seen, tables[0], planned.swa, plain.swa), (entries, tables[1], planned.main, plain.main)):
                x = mine[ints(table[b, rows // page], torch.long), ints(rows % page, torch.long)]
                y = theirs[ints(own[b].cpu().numpy()[rows // page], torch.long), ints(rows % page, torch.long)]
                assert torch.equal(x, y) and not x.isnan().any(), (step, b)
        done = (at + 1) % ratio == 0
        want = np.where(done, np.take_along_axis(tables[1], at // ratio // page, 1).astype(np.int64) * page + at // ratio % page, -1)
        np.testing.assert_array_equal(sides[1]["slots"].cpu().numpy().reshape(B, n), want)
        assert torch.equal(planned.out, plain.out) and torch.equal(planned.lse, plain.lse), step
        given = max(given, int(sides[0]["first"].max()))
        add.copy_(ints(rng.integers(2, n + 1, B)))
    assert given >= 2 and M.dsv4_read_device_flags() == 0
    for k in sides:
        assert int(k["count"]) + int((k["held"] - k["first"]).sum()) == k["pages"]
