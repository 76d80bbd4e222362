"""Grouped-query attention at the edges of what its header allows: page scales, hidden rows, caps, lengths."""
import numpy as np
import pytest
import torch

from gqa_cases import BF16_NAN, E4M3_NAN, Batch, bounds
from oracle import dsv4_oracle as O
from oracle import gqa_oracle as G
from test_gpu_gqa import M, check_attention, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------
# pages of very different scales
# ------------------------------------------------------------------------------------------------
SPREAD = [  # n, H, Hkv, D: 8, 16, 32 rows a kv head, and a long call
    (1, 8, 1, 128), (2, 16, 2, 64), (4, 16, 2, 128), (3, 10, 1, 64), (60, 4, 2, 128)]
SPREAD_IDS = [f"n{n}_g{H // k}_d{D}" for n, H, k, D in SPREAD]


def spread_batch(n, H, Hkv, D, kv=600, page=16):
    bt = Batch([n, 1], [kv, 47], H, Hkv, D, page, "e4m3", seed=n + D)
    for e in bt.exps:
        e[:] = 120
    return bt


@pytest.mark.parametrize("gap", [1, 4, 5, 16, 20, 24, 60, 100])
@pytest.mark.parametrize("n,H,Hkv,D", SPREAD, ids=SPREAD_IDS)
def test_scale_of_a_page_that_some_or_no_token_sees(M, n, H, Hkv, D, gap):
    """A page whose values' exponent lies `gap` above its neighbours': before every row that is seen; hidden from all
    tokens but the first; at either place of a pair of 16-row pages."""
    for page in (4, 5):
        for start in (np.full(n, 16 * page + 16), np.r_[0, np.full(n - 1, 16 * page + 16)], np.full(n, 16 * page + 19)):
            bt = spread_batch(n, H, Hkv, D)
            bt.exps[1][bt.table[0, page]] = 120 + gap
            check_attention(M, bt, kv_start=np.r_[start, 0])


@pytest.mark.parametrize("gap", [4, 5, 24, 60, 120])
@pytest.mark.parametrize("n,H,Hkv,D", SPREAD, ids=SPREAD_IDS)
def test_scale_of_a_page_without_weight(M, n, H, Hkv, D, gap):
    """Every row of such a page is seen, but its logits lie far below the others, or its codes are zeros."""
    for page in (8, 9):
        bt = spread_batch(n, H, Hkv, D)
        bt.q[:] = O.bf16_encode(np.ones(bt.q.shape))
        at = bt.table[0, page]
        bt.exps[0][:] = 127
        for p in bt.table[0, :38]:
            bt.caches[0][p] = np.where(bt.caches[0][p] == E4M3_NAN, E4M3_NAN, O.e4m3_encode(0.03125))
        bt.caches[0][at] = O.e4m3_encode(-30.0 if gap < 100 else -60.0)  # logits of -240 and less (-340 and less)
        bt.exps[1][at] = 120 + gap
        check_attention(M, bt)
        bt.caches[0][at] = O.e4m3_encode(0.03125)
        bt.caches[1][at] = 0
        check_attention(M, bt)


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("n", [1, 4, 60])
def test_scales_of_any_size_in_every_page(M, page, n):
    """Random exponents over 60 binary orders in every page."""
    bt = Batch([n, 1], [600, 333], 8, 2, 128, page, "e4m3", seed=page + n)
    g = np.random.default_rng(page)
    bt.exps[1][:] = g.integers(90, 150, bt.exps[1].shape)
    check_attention(M, bt)
    check_attention(M, bt, window=77, sink=np.linspace(-3, 3, 8))


# ------------------------------------------------------------------------------------------------
# rows that no token sees
# ------------------------------------------------------------------------------------------------
HIDDEN = [  # n, kv, window, kv_start of the sequence's first tokens (the rest: 0), first row that a token sees
    (2, 100, 50, [80, 0], 50), (2, 100, 0, [2 ** 30, 60], 60), (3, 130, 40, [2 ** 30, 2 ** 30, 0], 90),
    (4, 200, 33, [196, 170, 199, 180], 170), (1, 77, 30, [60], 60), (1, 77, 30, [5], 47),
    (60, 300, 50, [290, 250, 260], 194), (40, 300, 64, [2 ** 30] * 30 + [0] * 10, 227)]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n,kv,window,starts,first", HIDDEN, ids=[f"n{h[0]}_kv{h[1]}_w{h[2]}_{h[4]}" for h in HIDDEN])
def test_rows_before_the_first_seen_one_hold_nan(M, n, kv, window, starts, first, page, cache):
    """The first row that any token sees is the least over those that see something, of the later of the token's
    window and its kv_start; NaN in all rows before it changes no bit."""
    start = np.r_[starts, np.zeros(n - len(starts), np.int64), 3]
    pos = kv - n + np.arange(n)
    lo = np.maximum(start[:n], pos - window + 1 if window else 0)
    assert lo[lo <= pos].min() == first
    clean, bt = (Batch([n, 1], [kv, 20], 4, 2, 64, page, cache, seed=8) for _ in range(2))
    for j in range(first):
        for c in bt.caches:
            c[bt.table[0, j // page], :, j % page] = E4M3_NAN if cache == "e4m3" else BF16_NAN
    _, out, lse = run_attention(M, bt, window=window, kv_start=start)
    _, want, wlse = check_attention(M, clean, window=window, kv_start=start)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("n,kv,window,start", [(1, 100, 20, 0), (1, 101, 0, 81), (4, 700, 33, 0), (60, 300, 33, 0),
                                               (60, 900, 0, 700), (200, 500, 60, 0)])
def test_pages_before_the_first_seen_row_are_not_looked_at(M, n, kv, window, start, page, cache):
    """Entries of pages that lie before every token's window or start (a cache that lets go of them) may hold
    anything: not flagged, and no bit changes."""
    kv_start = np.r_[np.full(n, start), 0]
    first = max(start, kv - n - window + 1 if window else 0)
    clean, bt = (Batch([n, 1], [kv, 20], 4, 2, 64, page, cache, seed=8) for _ in range(2))
    _, want, wlse = check_attention(M, clean, window=window, kv_start=kv_start)
    for entry in (-1, 2 ** 31 - 1):
        bt.table[0, :first // page] = entry
        _, out, lse = run_attention(M, bt, window=window, kv_start=kv_start)
        assert M.dsv4_read_device_flags() == 0
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    if first // page < (kv - 1) // page:  # the page of the first seen row is
        bt.table[0, first // page] = -1
        run_attention(M, bt, window=window, kv_start=kv_start)
        assert M.dsv4_read_device_flags() == 1


# ------------------------------------------------------------------------------------------------
# capped scores
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("gain", [2.0 ** 90, 2.0 ** 40, 2.0 ** -40])
@pytest.mark.parametrize("cap", [12.0, 27.0, 30.0, 50.0, 500.0])
@pytest.mark.parametrize("n,causal", [(1, True), (60, True), (200, False)])
def test_capped_logits_from_end_to_end(M, n, causal, cap, gain, sink):
    """Rows whose logits lie at -cap in the first tiles, then at 0, then at +cap, over large and small values: the
    running softmax holds every weight in fp32 (2^100 over |v| times the rows seen is the range it promises).
    Bounds: those of the other calls, and the cap's own softcap * 2^-20."""
    bt = Batch([n, 3], [700, 300], 4, 2, 128, 64, "bf16", seed=3)
    bt.q[:] = O.bf16_encode(np.ones(bt.q.shape))
    bt.q[:, 1] = O.bf16_encode(-np.ones(bt.q.shape[2]))
    scale = 128 ** -0.5
    bt.caches[1][:] = np.where(bt.caches[1] == BF16_NAN, BF16_NAN,
                               O.bf16_encode(O.bf16_decode(bt.caches[1]).astype(np.float64) * gain))
    for b, kv in enumerate(bt.kv):
        for j in range(kv):
            z = (-4 if j < 300 else 0.01 * (j % 7) if j < 560 else 4) * cap
            bt.caches[0][bt.table[b, j // 64], :, j % 64] = O.bf16_encode(z / (128 * scale))
    kw = {"sink": cap * np.linspace(-1.5, 1, 4)} if sink else {}
    _, out, lse = run_attention(M, bt, softcap=cap, causal=causal, **kw)
    assert M.dsv4_read_device_flags() == 0
    want, wlse, mag, size = G.attention(bt.q64(), bt.caches, None, bt.table, bt.q_start, bt.kv, scale, causal=causal,
                                        softcap=cap, **kw)
    tol, ltol = bounds(mag, np.minimum(size, cap), want, wlse, False)
    off = cap * 2.0 ** -20
    tol, ltol = tol + mag * 2 * np.expm1(off), ltol + off
    # Beside a sink, the factor 2^(m - sink) of a row's sums is an fp32 number, 0 below 2^-126; the weights it stands for
    # are at most 2^20 above the reference m: each is then below 2^-106 of the total (here e^-100 = 2^-144).
    vmax = np.nanmax(np.abs(O.bf16_decode(bt.caches[1])).astype(np.float64))
    tol = tol + bt.max_kv * 2.0 ** -106 * vmax
    worst = np.max(np.abs(out.double().cpu().numpy() - want) / tol)
    assert worst <= 1, worst
    worst = np.max(np.abs(lse.double().cpu().numpy() - wlse) / ltol)
    assert worst <= 1, worst


# ------------------------------------------------------------------------------------------------
# very long sequences
# ------------------------------------------------------------------------------------------------
def long_run(M, n, H, kv, cache, page=256, D=128, kv_start=None, softcap=0.0, sink=None, out_dtype=torch.float32):
    """One kv head over kv rows that are one page again and again; the outputs and logsumexps, and the exact ones
    (each row of the page weighs as often as a token sees it) with the bounds' magnitudes."""
    bt = Batch([n], [page], H, 1, D, page, cache, seed=5)
    at = bt.table[0, 0]
    bt.table = np.full((1, kv // page), at, np.int32)
    bt.kv[:] = kv
    bt.max_kv = kv
    _, out, lse = run_attention(M, bt, kv_start=kv_start, softcap=softcap, sink=sink, out_dtype=out_dtype)
    assert M.dsv4_read_device_flags() == 0
    k, v = (G.rows_of(c, None if bt.exps is None else e, np.array([at]), 0, page)
            for c, e in zip(bt.caches, bt.exps or (None, None)))
    z = np.einsum("thd,jd->thj", bt.q64(), k) * D ** -0.5
    size = (np.einsum("thd,jd->thj", np.abs(bt.q64()), np.abs(k)) * D ** -0.5).max(-1)
    if softcap:
        z = softcap * np.tanh(z / softcap)

    def rows_up_to(x):
        return x[:, None] // page + (np.arange(page) < x[:, None] % page)

    count = rows_up_to(kv - n + np.arange(n) + 1) - (rows_up_to(kv_start) if kv_start is not None else 0)
    w = np.exp(z - z.max(-1, keepdims=True)) * count[:, None]
    total = w.sum(-1) + (0 if sink is None else np.exp(sink - z.max(-1)))
    want, mag = (np.einsum("thj,jd->thd", w / total[..., None], x) for x in (v, np.abs(v)))
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), want, z.max(-1) + np.log(total), mag, size


def test_a_piece_of_many_tiles_is_waited_for(M):
    """2^25 rows for a unit of 256 queries on each SM: a CTA's piece takes half a second, and no wait gives up."""
    out, lse, *_ = long_run(M, 304, 128, 2 ** 25, "bf16")
    assert (out != -3).all() and (lse != -3).all()


@pytest.mark.parametrize("kv", [2 ** 17, 2 ** 20, 2 ** 22, 2 ** 25])
@pytest.mark.parametrize("cache,n,H", [("bf16", 304, 128), ("bf16", 700, 128), ("bf16", 9, 40), ("e4m3", 9, 40), ("bf16", 1, 8),
                                        ("e4m3", 1, 8)])
def test_sums_over_many_rows(M, cache, n, H, kv):
    """As close as the sums over few rows."""
    out, lse, want, wlse, mag, size = long_run(M, n, H, kv, cache)
    tol, ltol = bounds(mag, size, want, wlse, False)
    worst = np.max(np.abs(out - want) / tol), np.max(np.abs(lse - wlse) / ltol)
    assert max(worst) <= 1, worst


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_sums_over_many_rows_of_some_tokens(M, softcap, D, out_dtype):
    """Tokens that see from 2^18 rows down to a few: of a unit's two row tiles one may go on for many runs without the
    other.  With a cap, its own softcap * 2^-20 more."""
    kv, n, H = 2 ** 20, 800, 96
    g = np.random.default_rng(7)
    start = kv - n + np.arange(n) - np.exp2(g.uniform(0, 18, n)).astype(np.int64)
    start[100:140] = kv - 5 * 2 ** 17 - 77
    start[300:303] = 0
    start[600:] = np.sort(start[600:])
    sink = np.linspace(-4, 14, H)
    out, lse, want, wlse, mag, size = long_run(M, n, H, kv, "bf16", D=D, kv_start=start, softcap=softcap, sink=sink,
                                               out_dtype=out_dtype)
    tol, ltol = bounds(mag, size, want, wlse, out_dtype == torch.bfloat16)
    off = softcap * 2.0 ** -20
    tol, ltol = tol + mag * 2 * np.expm1(off), ltol + off
    worst = np.max(np.abs(out - want) / tol), np.max(np.abs(lse - wlse) / ltol)
    assert max(worst) <= 1, worst


@pytest.mark.parametrize("cap", [20.0, 30.0, 50.0])
@pytest.mark.parametrize("n", [1, 60])
def test_capped_weight_of_one_row_is_not_rounded(M, n, cap):
    """A row far above the others in a token's first tile weighs a power of two, so the output is its value: the others
    together weigh under 600 e^-16 = 2^-13.8 of it, the sums and the division a few steps of 2^-23."""
    bt = Batch([n], [700], 8, 1, 128, 64, "bf16", seed=3)
    bt.q[:] = O.bf16_encode(np.linspace(1, 1.7, 8)[:, None] * np.ones(bt.q.shape))
    for j in range(700):
        z = 14.0 if j == 40 else -14.0     # caps of 20 and more leave at least 11.9 of it, and 16 between any two
        bt.caches[0][bt.table[0, j // 64], :, j % 64] = O.bf16_encode(z / 128 ** 0.5)
    _, out, _ = run_attention(M, bt, softcap=cap)
    v = O.bf16_decode(bt.caches[1][bt.table[0, 0], 0, 40]).astype(np.float64)
    big = np.abs(O.bf16_decode(bt.caches[1][bt.table[0]].view(np.uint16))).astype(np.float64)
    off = np.abs(out.double().cpu().numpy() - v)
    assert (off <= 2.0 ** -13 * np.nanmax(big) + 2.0 ** -20 * np.abs(v)).all(), off.max()
