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
