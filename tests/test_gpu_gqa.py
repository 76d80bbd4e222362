"""Grouped-query append and attention on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from gqa_cases import Batch, bounds, dev, host, strided
from oracle import dsv4_oracle as O
from oracle import gqa_oracle as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_v4_hybrid_gb300 as mod
    return mod


def cos_sin(n, rope_dim, seed=3):
    """Any table: the definition does not need cos^2 + sin^2 = 1."""
    return np.random.default_rng(seed).uniform(-1, 1, (n, rope_dim)).astype(np.float32)


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------
def run_append(M, bt, rope=None, first=0, halves=False, layout="hnd", with_q=True, in_place=False, device="cuda"):
    """Runs the append on the device and the oracle on copies; returns both sides' caches, exponents, queries."""
    kc, vc = (strided(dev(c), layout) for c in bt.caches)
    ke, ve = (None, None) if bt.exps is None else (dev(e) for e in bt.exps)
    qkv = torch.cat([dev(bt.q), dev(bt.k_new), dev(bt.v_new)], 1)      # rows of a fused projection
    q, k, v = qkv[:, :bt.H], qkv[:, bt.H:bt.H + bt.Hkv], qkv[:, bt.H + bt.Hkv:]
    q_out = q if in_place else torch.full((bt.T, bt.H, bt.D), -3.0, dtype=torch.bfloat16, device=device)
    p = M.gqa_append_params(k, v, kc, vc, dev(bt.table), dev(bt.q_start), dev(bt.kv), bt.max_q, k_scale=ke, v_scale=ve,
                            cos_sin=dev(rope), rope_first=first, rope_halves=halves, q=q if with_q else None,
                            q_out=q_out if with_q else None)
    M.dsv4_gqa_append(p)
    flags = M.dsv4_read_device_flags()
    want_c = [c.copy() for c in bt.caches]
    want_e = None if bt.exps is None else [e.copy() for e in bt.exps]
    G.append(O.bf16_decode(bt.k_new), O.bf16_decode(bt.v_new), want_c, want_e, bt.table, bt.q_start, bt.kv, rope, first,
             halves)
    got_c = [host(kc), host(vc)]
    got_e = None if ke is None else [host(ke), host(ve)]
    return p, flags, got_c, got_e, want_c, want_e, host(q_out)


def check_append(M, bt, rope=None, first=0, halves=False, **kw):
    _, flags, got_c, got_e, want_c, want_e, q_out = run_append(M, bt, rope, first, halves, **kw)
    assert flags == 0
    for c in range(2):
        if want_e is not None:
            np.testing.assert_array_equal(got_e[c], want_e[c])
        np.testing.assert_array_equal(got_c[c], want_c[c])
    if kw.get("with_q", True):
        live = int(bt.q_start[-1])
        want = np.stack([O.bf16_encode(G.rotate(O.bf16_decode(bt.q[t]), bt.kv[b] - bt.n[b] + t - bt.q_start[b], rope,
                                                first, halves))
                         for b in range(len(bt.n)) for t in range(bt.q_start[b], bt.q_start[b + 1])])
        np.testing.assert_array_equal(q_out[:live], want)
        rest = host(dev(bt.q))[live:] if kw.get("in_place") else O.bf16_encode(np.full((bt.T - live, bt.H, bt.D), -3.0))
        np.testing.assert_array_equal(q_out[live:], rest)


SHAPES = [  # n, kv, H, Hkv, D, page
    ([1], [1], 8, 2, 128, 64),
    ([1, 1, 1], [64, 65, 700], 16, 2, 128, 64),
    ([3, 0, 70, 1], [3, 5, 133, 16], 5, 1, 64, 16),
    ([200, 64, 1], [263, 64, 63], 6, 3, 128, 32),
    ([300, 2], [300, 258], 4, 4, 128, 256),
    ([129, 130], [129, 140], 3, 1, 64, 128),
    ([33, 1], [40, 257], 2, 2, 64, 256),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"n{max(s[0])}_h{s[2]}k{s[3]}_d{s[4]}_p{s[5]}")
def test_append_is_exact(M, shape, cache):
    n, kv, H, Hkv, D, page = shape
    bt = Batch(n, kv, H, Hkv, D, page, cache, seed=len(n) + D, pad=2)
    check_append(M, bt, cos_sin(max(kv), D))


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("D,first,rope", [(128, 64, 64), (128, 0, 32), (64, 8, 48), (128, 112, 16), (64, 0, 64), (128, 0, 0)])
def test_append_rotations(M, D, first, rope, halves):
    bt = Batch([5, 1, 40], [9, 300, 64], 5, 2, D, 32, "e4m3", seed=first)
    check_append(M, bt, cos_sin(300, rope) if rope else None, first, halves)
    check_append(M, Batch([2, 3], [2, 70], 17, 1, D, 16, "bf16", seed=first + 1), cos_sin(70, rope) if rope else None, first,
                 halves, in_place=True)


@pytest.mark.parametrize("layout", ["nhd", "wide"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_cache_layouts(M, layout, cache):
    bt = Batch([3, 90], [10, 90], 4, 3, 128, 32, cache, seed=7)
    check_append(M, bt, cos_sin(90, 128), layout=layout, with_q=False)


@pytest.mark.parametrize("gain", [2.0 ** -40, 0.0, 1.0, 2.0 ** 12, 2.0 ** 100, 2.0 ** 125])
def test_append_growing_and_extreme_scales(M, gain):
    """New rows far smaller and far larger than the page's earlier ones: exponents and re-encoded codes exact."""
    bt = Batch([2, 1, 20], [40, 33, 35], 2, 2, 128, 32, "e4m3", seed=11)
    for x in (bt.k_new, bt.v_new):
        x[:] = O.bf16_encode(O.bf16_decode(x).astype(np.float64) * gain)
    check_append(M, bt)


def test_append_all_zero_rows_then_values(M):
    """A page begun with zeros takes the next rows' exponent."""
    bt = Batch([1], [1], 1, 1, 64, 16, "e4m3", seed=1)
    bt.k_new[:] = 0
    p, flags, got_c, got_e, want_c, want_e, _ = run_append(M, bt)
    assert flags == 0 and got_e[0][bt.table[0, 0], 0] == 0 and not got_c[0][bt.table[0, 0], 0, 0].any()
    b2 = Batch([1], [2], 1, 1, 64, 16, "e4m3", seed=1)
    b2.caches, b2.exps, b2.table = want_c, want_e, bt.table
    check_append(M, b2)


def test_append_infinities_saturate(M):
    bt = Batch([2], [2], 1, 1, 64, 16, "e4m3", seed=2)
    bt.k_new[0, 0, 5] = 0x7F80
    bt.v_new[1, 0, 3] = 0x7FC0
    _, flags, got_c, got_e, _, want_e, _ = run_append_device_only(M, bt)
    page = bt.table[0, 0]
    assert flags == 0
    assert got_e[0][page, 0] == 120 + 127 and got_c[0][page, 0, 0, 5] == 0x7E
    assert got_c[1][page, 0, 1, 3] & 0x7F == 0x7F
    assert np.isfinite(O.e4m3_decode(got_c[1][page, 0, 0])).all()


def run_append_device_only(M, bt):
    kc, vc = dev(bt.caches[0]), dev(bt.caches[1])
    ke, ve = dev(bt.exps[0]), dev(bt.exps[1])
    p = M.gqa_append_params(dev(bt.k_new), dev(bt.v_new), kc, vc, dev(bt.table), dev(bt.q_start), dev(bt.kv), bt.max_q,
                            k_scale=ke, v_scale=ve)
    M.dsv4_gqa_append(p)
    return p, M.dsv4_read_device_flags(), [host(kc), host(vc)], [host(ke), host(ve)], None, None, None


def test_append_skips_and_flags_bad_sequences(M):
    """Bad table entries, lengths over the table or the rotation's table, too many new tokens, kv_len < n: flagged,
    nothing stored for them; the other sequences as ever."""
    bt = Batch([2, 3, 2, 1], [40, 33, 8, 5], 2, 1, 128, 16, "e4m3", seed=4)
    cs = cos_sin(40, 128)
    good = run_append(M, bt, cs)
    for what in ("page", "negative", "kv", "max_q", "max_pos"):
        b2 = Batch([2, 3, 2, 1], [40, 33, 8, 5], 2, 1, 128, 16, "e4m3", seed=4)
        table, kv, q_start, rope, max_q = b2.table.copy(), b2.kv.copy(), b2.q_start.copy(), cs, b2.max_q
        if what == "page":
            table[1, 2] = b2.caches[0].shape[0]
        elif what == "negative":
            table[1, 2] = -1
        elif what == "kv":
            kv[1] = 2
        elif what == "max_q":
            max_q = 2
        else:
            kv[1] = 41
        kc, vc, ke, ve = dev(b2.caches[0]), dev(b2.caches[1]), dev(b2.exps[0]), dev(b2.exps[1])
        p = M.gqa_append_params(dev(b2.k_new), dev(b2.v_new), kc, vc, dev(table), dev(q_start), dev(kv), max_q, k_scale=ke,
                                v_scale=ve, cos_sin=dev(rope))
        M.dsv4_gqa_append(p)
        assert M.dsv4_read_device_flags() == 1, what
        got = host(kc)
        mine = [x for x in bt.table[1, :3]]
        others = [x for x in range(got.shape[0]) if x not in mine]
        np.testing.assert_array_equal(got[others], good[2][0][others])
        if what in ("kv", "max_q", "max_pos"):
            np.testing.assert_array_equal(got[mine], bt.caches[0][mine])


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def run_attention(M, bt, scale=None, layout="hnd", out_dtype=torch.float32, max_q=None, max_kv=None, stream=None, **opt):
    scale = bt.D ** -0.5 if scale is None else scale
    kc, vc = (strided(dev(c), layout) for c in bt.caches)
    ke, ve = (None, None) if bt.exps is None else (dev(e) for e in bt.exps)
    buf = torch.zeros((bt.T, bt.H + 3, bt.D), dtype=torch.bfloat16, device="cuda")
    buf[:, 1:bt.H + 1] = dev(bt.q)
    out = torch.full((bt.T, bt.H, bt.D), -3.0, dtype=out_dtype, device="cuda")
    lse = torch.full((bt.T, bt.H), -3.0, device="cuda")
    arrays = {k: dev(np.asarray(v, np.int32 if k in ("prefix_len", "kv_start") else np.float32))
              for k, v in opt.items() if k in ("prefix_len", "kv_start", "slopes", "sink") and v is not None}
    plain = {k: v for k, v in opt.items() if k in ("causal", "window", "softcap")}
    p = M.gqa_attention_params(buf[:, 1:bt.H + 1], kc, vc, dev(bt.table), dev(bt.q_start), dev(bt.kv),
                               bt.max_q if max_q is None else max_q, bt.max_kv if max_kv is None else max_kv, scale, out,
                               lse=lse, k_scale=ke, v_scale=ve, **arrays, **plain)
    ws = torch.full((M.dsv4_gqa_attention_workspace_bytes(p),), 255, dtype=torch.uint8, device="cuda")
    M.gqa_set_workspace(p, ws)
    M.dsv4_gqa_attention(p, stream)
    return p, out, lse


def check_attention(M, bt, out_dtype=torch.float32, flags=0, **kw):
    p, out, lse = run_attention(M, bt, out_dtype=out_dtype, **kw)
    assert M.dsv4_read_device_flags() == flags
    opt = {k: v for k, v in kw.items() if k not in ("scale", "layout", "max_q", "max_kv", "stream")}
    scale = kw.get("scale", bt.D ** -0.5)
    want, wlse, mag, size = G.attention(bt.q64(), bt.caches, bt.exps, bt.table, bt.q_start, bt.kv, scale, **opt)
    live = int(bt.q_start[-1])
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (got[live:] == -3).all() and (glse[live:] == -3).all()
    tol, ltol = bounds(mag, size, want, wlse, out_dtype == torch.bfloat16)
    got, glse, want, wlse, tol, ltol = (x[:live] for x in (got, glse, want, wlse, tol, ltol))
    np.testing.assert_array_equal(np.isneginf(glse), np.isneginf(wlse))
    fin = np.isfinite(wlse)
    assert np.isfinite(got).all() and np.isfinite(glse[fin]).all()
    off = np.abs(glse[fin] - wlse[fin]) / ltol[fin]
    assert off.max(initial=0.0) <= 1, off.max()
    worst = np.max(np.abs(got - want) / tol, initial=0.0)
    assert worst <= 1, worst
    assert (got[~fin] == 0).all()
    return p, out, lse


ATT_SHAPES = [  # n, kv, H, Hkv, D, page
    ([1], [1], 8, 8, 128, 64),
    ([1, 1, 1, 1], [1, 63, 64, 777], 16, 2, 128, 64),
    ([1, 0, 1], [130, 7, 2049], 8, 1, 64, 16),
    ([4, 2, 3], [4, 150, 900], 16, 2, 128, 32),
    ([2, 1], [500, 31], 12, 4, 64, 128),
    ([1, 1], [300, 257], 20, 1, 128, 256),
    ([4, 4], [200, 4], 64, 8, 128, 64),
    ([17, 5, 0, 1], [17, 200, 3, 90], 6, 2, 128, 64),
    ([65, 129], [300, 129], 5, 1, 128, 16),
    ([200], [456], 3, 3, 64, 32),
    ([33, 40], [33, 555], 14, 2, 64, 256),
    ([300], [300], 8, 2, 128, 128),
]
IDS = [f"n{max(s[0])}_kv{max(s[1])}_h{s[2]}k{s[3]}_d{s[4]}_p{s[5]}" for s in ATT_SHAPES]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", ATT_SHAPES, ids=IDS)
def test_attention_causal(M, shape, cache):
    n, kv, H, Hkv, D, page = shape
    check_attention(M, Batch(n, kv, H, Hkv, D, page, cache, seed=D + page, pad=1))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [ATT_SHAPES[i] for i in (1, 3, 7, 8, 10)], ids=[IDS[i] for i in (1, 3, 7, 8, 10)])
def test_attention_every_option_together(M, shape, cache, out_dtype):
    n, kv, H, Hkv, D, page = shape
    bt = Batch(n, kv, H, Hkv, D, page, cache, seed=5, qscale=3.0, pad=3)
    g = np.random.default_rng(9)
    start = np.concatenate([np.maximum(0, k - m + np.arange(m) - g.integers(0, 60)) for m, k in zip(n, kv)] + [[0] * 3])
    check_attention(M, bt, out_dtype=out_dtype, softcap=8.0, window=100, slopes=g.uniform(0, 0.3, H),
                    sink=g.standard_normal(H), prefix_len=[min(k, 40) for k in kv], kv_start=start)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("opt", [dict(softcap=5.0), dict(window=1), dict(window=70), dict(causal=False), dict(sink=True),
                                 dict(slopes=True), dict(prefix=100), dict(window=30, causal=False),
                                 dict(softcap=1e-3), dict(scale=0.0), dict(scale=-0.2)],
                         ids=lambda o: "_".join(o))
def test_attention_single_options(M, opt, cache):
    for n, kv in (([1, 3], [500, 129]), ([150, 20], [310, 20])):
        bt = Batch(n, kv, 8, 2, 128, 64, cache, seed=21, qscale=2.0)
        o = dict(opt)
        if o.pop("sink", None):
            o["sink"] = np.linspace(-30, 30, 8)
        if o.pop("slopes", None):
            o["slopes"] = 2.0 ** -np.arange(8)
        if "prefix" in o:
            o["prefix_len"] = [min(k, o["prefix"]) for k in kv]
            del o["prefix"]
        check_attention(M, bt, **o)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("n,kv", [([2, 1], [90, 40]), ([70, 40], [90, 40])])
def test_tokens_that_see_nothing(M, n, kv, sink):
    """kv_start behind the token, an empty window through kv_start, and a document that begins at the last token:
    zeros and lse = sink."""
    bt = Batch(n, kv, 4, 2, 128, 32, "e4m3", seed=2)
    pos = np.concatenate([np.arange(k - m, k) for m, k in zip(n, kv)])
    start = pos.copy()
    start[::2] += 1                        # every other token sees nothing
    start[-1] = 2 ** 30
    kw = {"sink": np.array([0.5, -2.0, -np.inf, 3.0])} if sink else {}
    check_attention(M, bt, kv_start=start, **kw)


def test_rows_behind_and_before_hold_nan(M):
    """NaN in the rows before every token's window, behind kv_len and in unused pages."""
    for n, kv in (([1, 2], [400, 100]), ([40, 33], [400, 300])):
        for cache in ("bf16", "e4m3"):
            bt = Batch(n, kv, 4, 1, 64, 32, cache, seed=8)
            w = 50
            for b in range(2):
                for j in range(0, kv[b] - n[b] - w + 1):
                    for c in bt.caches:
                        c[bt.table[b, j // 32], :, j % 32] = 0x7F if cache == "e4m3" else 0x7FC0
            clean = Batch(n, kv, 4, 1, 64, 32, cache, seed=8)
            p, out, lse = run_attention(M, bt, window=w)
            _, out2, lse2 = check_attention(M, clean, window=w)
            assert torch.isfinite(out).all()
            assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", ["nhd", "wide"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_cache_layouts(M, layout, cache):
    check_attention(M, Batch([1, 2], [300, 65], 8, 2, 128, 64, cache, seed=1), layout=layout)
    check_attention(M, Batch([100, 20], [100, 165], 8, 2, 64, 16, cache, seed=1), layout=layout)


def test_attention_scale_spread_over_pages(M):
    """Pages whose exponents lie far apart, and the smallest and largest useful ones."""
    for n, kv in (([1], [600]), ([60], [600])):
        bt = Batch(n, kv, 4, 2, 128, 64, "e4m3", seed=6)
        used = bt.table[0, :10]
        for i, page in enumerate(used):
            bt.exps[0][page] = 110 + i % 4
            bt.exps[1][page] = (60, 120, 121, 127, 150, 119, 20, 122, 121, 140)[i]
        check_attention(M, bt)


def test_attention_large_logits(M):
    """Logits of some hundreds, of both signs: the running maximum moves."""
    for n, kv in (([1, 1], [900, 901]), ([130], [700])):
        check_attention(M, Batch(n, kv, 8, 2, 128, 64, "bf16", seed=3, qscale=60.0))
        check_attention(M, Batch(n, kv, 8, 2, 128, 64, "e4m3", seed=3, qscale=60.0))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("at", [{70: 12.0}, {200: 14.0, 230: 20.0, 310: 60.0}, {250: 75.0, 400: 160.0}, {215: 300.0}, {0: 90.0},
                                {500: -200.0, 330: 90.0, 459: 91.0, 460: 170.0}], ids=lambda a: "_".join(map(str, a)))
def test_attention_logits_that_jump(M, at, cache):
    """Flat logits but for a few rows far above (or below) them: the reference of the running softmax moves late, by
    little, by much and in the second half of a tile."""
    for n, kv in (([1], [600]), ([60, 3], [600, 599])):
        bt = Batch(n, kv, 4, 2, 128, 64, cache, seed=3)
        bt.q[:] = O.bf16_encode(np.ones(bt.q.shape))
        bt.q[:, 1] = O.bf16_encode(-np.ones(bt.q.shape[2]))
        if cache == "e4m3":
            bt.exps[0][:] = 127
        for b in range(len(n)):
            for j in range(kv[b]):
                v = at.get(j, 0.01 * (j % 7)) * 128 ** 0.5 / 128
                bt.caches[0][bt.table[b, j // 64], :, j % 64] = O.bf16_encode(v) if cache == "bf16" else O.e4m3_encode(v)
        check_attention(M, bt)


@pytest.mark.parametrize("cap", [0.5, 30.0])
def test_attention_capped_within_and_beyond(M, cap):
    """Logits well inside the cap, around it and far beyond it (the two forms of the tanh)."""
    for n, kv in (([1, 4], [300, 129]), ([90, 20], [310, 20])):
        for gain in (0.02, 1.0, 40.0):
            check_attention(M, Batch(n, kv, 8, 2, 128, 64, "bf16", seed=5, qscale=gain * cap), softcap=cap)


def test_attention_bounds_larger_than_the_batch(M):
    bt = Batch([1, 3], [300, 65], 8, 2, 128, 64, "e4m3", seed=1)
    check_attention(M, bt, max_q=4, max_kv=100000)
    check_attention(M, bt, max_q=300, max_kv=301)


def test_attention_flags_bad_pages_and_sequences(M):
    for n, kv in (([1, 2, 1], [300, 65, 20]), ([100, 70, 20], [300, 165, 20])):
        for cache in ("bf16", "e4m3"):
            bt = Batch(n, kv, 4, 2, 128, 64, cache, seed=4)
            good = check_attention(M, bt)[1]
            want, wlse, mag, size = G.attention(bt.q64(), bt.caches, bt.exps, bt.table, bt.q_start, bt.kv, bt.D ** -0.5)
            # (where the rows are cut depends on the whole batch, so another batch gives other roundings: both
            # results are within tol of the exact ones)
            tol = torch.from_numpy(bounds(mag, size, want, wlse, False)[0]).cuda()

            def same(out, t0, t1):
                return bool(((out[t0:t1] - good[t0:t1]).abs().double() <= 2 * tol[t0:t1]).all())

            for entry in (-1, bt.caches[0].shape[0], 2 ** 31 - 1):
                b2 = Batch(n, kv, 4, 2, 128, 64, cache, seed=4)
                b2.table[0, 1] = entry
                _, out, _ = run_attention(M, b2)
                assert M.dsv4_read_device_flags() == 1
                assert torch.isfinite(out).all()
                t1 = int(bt.q_start[1])
                assert same(out, t1, bt.T)
                assert not torch.equal(out[:t1], good[:t1])
            for what in ("kv", "max_kv", "max_q"):
                b2 = Batch(n, kv, 4, 2, 128, 64, cache, seed=4)
                kw = {}
                if what == "kv":
                    b2.kv[0] = n[0] - 1
                elif what == "max_kv":
                    kw["max_kv"] = 299
                else:
                    kw["max_q"] = max(n) - 1
                _, out, lse = run_attention(M, b2, **kw)
                assert M.dsv4_read_device_flags() == 1
                bad = int(np.argmax(n)) if what == "max_q" else 0
                for b in range(3):
                    t0, t1 = int(bt.q_start[b]), int(bt.q_start[b + 1])
                    assert ((out[t0:t1] == -3).all() if b == bad else same(out, t0, t1)), what


def test_attention_is_repeatable_and_replays(M):
    """Twice the same bits; captured and replayed with new inputs; another stream."""
    for n, kv in (([1] * 5, [3000, 40, 900, 77, 2000]), ([90, 5], [1000, 5])):
        bt = Batch(n, kv, 16, 2, 128, 64, "e4m3", seed=14)
        p, out, lse = run_attention(M, bt)
        first = out.clone()
        M.dsv4_gqa_attention(p)
        assert torch.equal(out, first)
        out.fill_(7)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            M.dsv4_gqa_attention(p)
        s.synchronize()
        assert torch.equal(out, first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.dsv4_gqa_attention(p)
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        p.tensors[0].mul_(-1)                 # the queries, in place
        M.dsv4_gqa_attention(p)
        again = out.clone()
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again) and not torch.equal(out, first)
        assert M.dsv4_read_device_flags() == 0


# ------------------------------------------------------------------------------------------------
# the two together, as a decode loop uses them
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_prompt_then_decode(M, cache):
    """Two prompts stored and attended in one call, in chunks for one of them, then single tokens, each step against
    the oracle on the oracle's own caches; codes stay equal throughout."""
    H, Hkv, D, page, scale = 8, 2, 64, 16, 0.2
    g = np.random.default_rng(0)
    steps = [([70, 9], [70, 9]), ([30, 9], [100, 18])] + [([1, 1], [101 + i, 19 + i]) for i in range(3)] + [([4, 0], [107, 21])]
    pages = 12
    order = g.permutation(pages)
    table = np.full((2, 7), -1, np.int32)
    table[0], table[1, :5] = order[:7], order[7:]
    dt = np.uint16 if cache == "bf16" else np.uint8
    want_c = [np.zeros((pages, Hkv, page, D), dt) for _ in range(2)]
    want_e = None if cache == "bf16" else [np.zeros((pages, Hkv), np.uint8) for _ in range(2)]
    kc, vc = dev(want_c[0]), dev(want_c[1])
    ke, ve = (None, None) if want_e is None else (dev(want_e[0]), dev(want_e[1]))
    cs = cos_sin(128, D)
    dtab, dcs = dev(table), dev(cs)
    for i, (n, kv) in enumerate(steps):
        T = sum(n)
        grow = 1.0 + i                        # later rows larger: exponents grow inside pages
        x = O.bf16_encode(g.standard_normal((T, H + 2 * Hkv, D)) * grow)
        qkv = dev(x)
        q_start, kvl = np.concatenate([[0], np.cumsum(n)]).astype(np.int32), np.asarray(kv, np.int32)
        dq, dkv = dev(q_start), dev(kvl)
        q_rot = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        ap = M.gqa_append_params(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, dtab, dq, dkv, max(n), k_scale=ke,
                                 v_scale=ve, cos_sin=dcs, q=qkv[:, :H], q_out=q_rot)
        out = torch.empty((T, H, D), device="cuda")
        at = M.gqa_attention_params(q_rot, kc, vc, dtab, dq, dkv, max(n), max(kv), scale, out, k_scale=ke, v_scale=ve)
        M.gqa_set_workspace(at, torch.empty(M.dsv4_gqa_attention_workspace_bytes(at), dtype=torch.uint8, device="cuda"))
        M.dsv4_gqa_append(ap)
        M.dsv4_gqa_attention(at)
        assert M.dsv4_read_device_flags() == 0
        xf = O.bf16_decode(x)
        G.append(xf[:, H:H + Hkv], xf[:, H + Hkv:], want_c, want_e, table, q_start, kvl, cs)
        np.testing.assert_array_equal(host(kc), want_c[0])
        np.testing.assert_array_equal(host(vc), want_c[1])
        q64 = O.bf16_decode(host(q_rot)).astype(np.float64)
        want, wlse, mag, size = G.attention(q64, want_c, want_e, table, q_start, kvl, scale)
        tol, _ = bounds(mag, size, want, wlse, False)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all(), i


# ------------------------------------------------------------------------------------------------
# calls at the edges of what is allowed
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,D,n", [(8, 2, 64, 1), (12, 1, 128, 1), (8, 1, 64, 3)])
def test_attention_of_more_sequences_than_the_list_holds(M, H, Hkv, D, n, cache):
    """Over 1024 sequences a CTA takes a whole (sequence, kv head); 8, 12 and 24 rows a kv head, empty ones between."""
    g = np.random.default_rng(3)
    count = 1100
    ns = np.where(g.random(count) < 0.9, 0, n)
    ns[[0, 1023, 1024, count - 1]] = n
    kv = np.where(ns > 0, n + g.integers(0, 150, count), g.integers(0, 3, count))
    check_attention(M, Batch(ns, kv, H, Hkv, D, 16, cache, seed=1), sink=np.linspace(-1, 1, H))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_long_attention_of_more_units_than_the_list_holds(M, cache):
    """Over 8192 units of 256 rows a CTA takes a whole one, whatever the lengths."""
    g = np.random.default_rng(4)
    count = 2100
    ns = np.where(g.random(count) < 0.99, 0, 40)
    ns[[0, count - 1]] = 90
    kv = np.where(ns > 0, ns + g.integers(0, 150, count), g.integers(0, 3, count))
    check_attention(M, Batch(ns, kv, 4, 2, 64, 32, cache, seed=1), max_q=600)


@pytest.mark.parametrize("group", [3, 5, 7, 9, 48, 128, 200])
@pytest.mark.parametrize("D", [64, 128])
def test_long_attention_of_odd_groups(M, group, D):
    """Query tiles whose 128 rows do not hold whole tokens, or less than one."""
    check_attention(M, Batch([40, 3], [50, 200], group, 1, D, 64, "bf16", seed=group))


@pytest.mark.parametrize("group", [3, 5, 7, 9, 11, 15, 20, 31, 32])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_single_token_attention_of_odd_groups(M, group, cache):
    check_attention(M, Batch([1, 1, 0, 1], [1, 333, 0, 64], 2 * group, 2, 128, 32, cache, seed=group))


@pytest.mark.parametrize("n,kv", [([2, 1, 0], [90, 40, 0]), ([70, 0, 40], [90, 0, 400])])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_padding_tokens_may_hold_anything(M, n, kv, cache):
    """NaN in the padding's queries, keys and values; its outputs stay as they were."""
    bt = Batch(n, kv, 8, 2, 64, 32, cache, seed=6, pad=200)
    live = int(bt.q_start[-1])
    bt.q[live:] = bt.k_new[live:] = bt.v_new[live:] = 0x7FC0
    check_append(M, bt, cos_sin(400, 64))
    check_attention(M, bt)


@pytest.mark.parametrize("n,kv", [([4, 1], [100, 70]), ([40, 33], [100, 70])])
def test_one_query_for_every_token_and_head(M, n, kv):
    """Queries of stride 0: one row, read by all."""
    bt = Batch(n, kv, 4, 2, 64, 32, "e4m3", seed=6)
    bt.q[:] = bt.q[:1, :1]
    kc, vc, ke, ve = dev(bt.caches[0]), dev(bt.caches[1]), dev(bt.exps[0]), dev(bt.exps[1])
    out = torch.empty((bt.T, 4, 64), device="cuda")
    q = dev(bt.q[:1, :1]).expand(bt.T, 4, 64)
    p = M.gqa_attention_params(q, kc, vc, dev(bt.table), dev(bt.q_start), dev(bt.kv), bt.max_q, bt.max_kv, 0.125, out,
                               k_scale=ke, v_scale=ve)
    M.gqa_set_workspace(p, torch.empty(M.dsv4_gqa_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda"))
    M.dsv4_gqa_attention(p)
    assert M.dsv4_read_device_flags() == 0
    want, wlse, mag, size = G.attention(bt.q64(), bt.caches, bt.exps, bt.table, bt.q_start, bt.kv, 0.125)
    assert (np.abs(out.double().cpu().numpy() - want) <= bounds(mag, size, want, wlse, False)[0]).all()


@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_caches_and_positions_past_32_bits(M, n, cache):
    """Pages whose offsets pass 2^32 elements, at positions beyond 2^24 (odd ones, which fp32 does not hold), in a window:
    append, then attention with distance bias, against the oracle on the sequence's last pages."""
    H, Hkv, D, page, pages, W = 4, 1, 128, 256, 140000, 300
    e4m3 = cache == "e4m3"
    dt = torch.uint8 if e4m3 else torch.bfloat16
    kc, vc = (torch.empty((pages, Hkv, page, D), dtype=dt, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 32
    base = 78200 * page                                   # 20,019,200 rows before those that are looked at
    kv = base + 3 * page + 77                             # the window and the new rows lie in four pages
    mine = [pages - 1, 5, pages - 3, pages - 2]
    table = np.full((1, base // page + 4), -1, np.int32)
    table[0, -4:] = mine
    small = Batch([n], [kv - base], H, Hkv, D, page, cache, seed=3)
    g = np.random.default_rng(1)
    at = torch.tensor(mine, device="cuda")
    fill, exps = [], None
    for c in (kc, vc):
        x = O.bf16_encode(g.standard_normal((4, Hkv, page, D)))
        if e4m3:
            x = O.e4m3_encode(np.clip(g.standard_normal((4, Hkv, page, D)) * 100, -448, 448))
        fill.append(x)
        c[at] = dev(x)
    dev_e = [None, None]
    if e4m3:
        exps = [g.integers(117, 123, (4, Hkv)).astype(np.uint8) for _ in range(2)]
        dev_e = [torch.zeros((pages, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2)]
        for d, e in zip(dev_e, exps):
            d[at] = dev(e)
    tab, qs, kvl = dev(table), dev(small.q_start), dev(np.array([kv], np.int32))
    ap = M.gqa_append_params(dev(small.k_new), dev(small.v_new), kc, vc, tab, qs, kvl, n, k_scale=dev_e[0], v_scale=dev_e[1])
    M.dsv4_gqa_append(ap)
    assert M.dsv4_read_device_flags() == 0
    local = np.arange(4, dtype=np.int32)[None]
    local_kv = np.array([kv - base], np.int32)
    G.append(O.bf16_decode(small.k_new), O.bf16_decode(small.v_new), fill, exps, local, small.q_start, local_kv)
    for c, want in zip((kc, vc), fill):
        got = c[at]
        np.testing.assert_array_equal(host(got), want)
    out = torch.empty((n, H, D), device="cuda")
    slopes = np.array([2.0, 0.5, 0.25, 0.0])
    p = M.gqa_attention_params(dev(small.q), kc, vc, tab, qs, kvl, n, kv, 0.1, out, k_scale=dev_e[0], v_scale=dev_e[1],
                               window=W, slopes=dev(slopes.astype(np.float32)))
    size = M.dsv4_gqa_attention_workspace_bytes(p)
    M.gqa_set_workspace(p, torch.empty(size, dtype=torch.uint8, device="cuda"))
    M.dsv4_gqa_attention(p)
    assert M.dsv4_read_device_flags() == 0
    want, wlse, mag, size = G.attention(small.q64(), fill, exps, local, small.q_start, local_kv, 0.1, window=W, slopes=slopes)
    tol = bounds(mag, size, want, wlse, False)[0]
    worst = (np.abs(out.double().cpu().numpy() - want) / tol).max()
    assert worst <= 1, worst


def test_append_skips_lengths_over_two_to_thirty(M):
    bt = Batch([1, 1], [20, 9], 2, 1, 64, 16, "bf16", seed=3)
    kv = bt.kv.copy()
    kv[0] = 2 ** 30 + 1
    kc, vc = dev(bt.caches[0]), dev(bt.caches[1])
    p = M.gqa_append_params(dev(bt.k_new), dev(bt.v_new), kc, vc, dev(bt.table), dev(bt.q_start), dev(kv), 1)
    M.dsv4_gqa_append(p)
    assert M.dsv4_read_device_flags() == 1
    got = host(kc)
    np.testing.assert_array_equal(got[bt.table[0]], bt.caches[0][bt.table[0]])
    np.testing.assert_array_equal(got[bt.table[1, 0], :, 8], bt.k_new[1])


def test_two_streams_with_workspaces_of_their_own(M):
    """A long and a short call at once, twenty times over: the bits of the calls one after the other."""
    runs = []
    for n, kv in (([1] * 6, [3000, 40, 900, 77, 2000, 1]), ([90, 33], [1500, 700]), ([300, 2], [300, 900])):
        bt = Batch(n, kv, 16, 2, 128, 64, "e4m3", seed=14)
        p, out, _ = run_attention(M, bt)
        runs.append((p, out, out.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for p, out, _, s in runs:
            with torch.cuda.stream(s):
                out.fill_(7)
                M.dsv4_gqa_attention(p)
    torch.cuda.synchronize()
    for _, out, want, _ in runs:
        assert torch.equal(out, want)
    assert M.dsv4_read_device_flags() == 0


@pytest.mark.parametrize("n,max_q", [(1, 1), (4, 4), (40, 40)])
def test_captured_steps_replay_with_other_lengths(M, n, max_q):
    """Append and attention captured with no eager call before; the lengths, tables and rows change between replays."""
    H, Hkv, D, page = 8, 2, 128, 32
    a = Batch([n, n], [200, 130], H, Hkv, D, page, "e4m3", seed=1)
    b = Batch([n, 0], [55, 64], H, Hkv, D, page, "e4m3", seed=2, pad=n)
    width, pages = 8, 24
    tab = torch.zeros((2, width), dtype=torch.int32, device="cuda")
    qs, kvl = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ke, ve = (torch.zeros((pages, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    x = torch.zeros((2 * n, H + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    rot = torch.zeros((2 * n, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((2 * n, H, D), device="cuda")
    rope = cos_sin(300, D)
    ap = M.gqa_append_params(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, tab, qs, kvl, max_q, k_scale=ke, v_scale=ve,
                             cos_sin=dev(rope), q=x[:, :H], q_out=rot)
    at = M.gqa_attention_params(rot, kc, vc, tab, qs, kvl, max_q, width * page, 0.1, out, k_scale=ke, v_scale=ve)
    M.gqa_set_workspace(at, torch.empty(M.dsv4_gqa_attention_workspace_bytes(at), dtype=torch.uint8, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.dsv4_gqa_append(ap)
        M.dsv4_gqa_attention(at)
    for bt in (a, b, a):
        tab.fill_(-1)
        tab[:, :bt.table.shape[1]] = dev(bt.table)
        qs.copy_(dev(bt.q_start))
        kvl.copy_(dev(bt.kv))
        for c, e, hc, he in zip((kc, vc), (ke, ve), bt.caches, bt.exps):
            c[:len(hc)] = dev(hc)
            e[:len(he)] = dev(he)
        x.copy_(torch.cat([dev(bt.q), dev(bt.k_new), dev(bt.v_new)], 1))
        out.fill_(-3)
        g.replay()
        assert M.dsv4_read_device_flags() == 0
        caches, exps = [c.copy() for c in bt.caches], [e.copy() for e in bt.exps]
        G.append(O.bf16_decode(bt.k_new), O.bf16_decode(bt.v_new), caches, exps, bt.table, bt.q_start, bt.kv, rope)
        for c, want in zip((kc, vc), caches):
            np.testing.assert_array_equal(host(c)[:len(want)], want)
        want, wlse, mag, size = G.attention(O.bf16_decode(host(rot)).astype(np.float64), caches, exps, bt.table, bt.q_start,
                                            bt.kv, 0.1)
        live = int(bt.q_start[-1])
        tol = bounds(mag, size, want, wlse, False)[0]
        got = out.double().cpu().numpy()
        assert (np.abs(got - want)[:live] <= tol[:live]).all()
        assert (got[live:] == -3).all()


@pytest.mark.parametrize("n,kv", [([1, 3], [300, 65]), ([60, 70], [300, 70])])
@pytest.mark.parametrize("cap", [300.0, 1000.0])
def test_attention_wide_caps(M, n, kv, cap):
    """Caps far above the logits: off by softcap * 2^-22 more than the bounds, which the weights feel twice."""
    bt = Batch(n, kv, 8, 2, 128, 64, "bf16", seed=5, qscale=2.0)
    _, out, _ = run_attention(M, bt, softcap=cap)
    want, wlse, mag, size = G.attention(bt.q64(), bt.caches, bt.exps, bt.table, bt.q_start, bt.kv, bt.D ** -0.5, softcap=cap)
    tol = bounds(mag, size, want, wlse, False)[0] + mag * 2 * np.expm1(cap * 2.0 ** -22)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert M.dsv4_read_device_flags() == 0
