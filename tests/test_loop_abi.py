"""The calls around the layers: symbols, struct layouts, refusals and frequencies, without a GPU; and the
oracle's own pins."""
import ctypes as C
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import loop_oracle as L
from test_gqa_abi import abi  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dsv4_loop.h")


def test_exports_and_struct_layout(abi, tmp_path):  # noqa: F811
    names = set(re.findall(r"^\s*int\s+(dsv4_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(abi.LOOP_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", abi.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\bT (dsv4_\w+)", out))
    structs = {"dsv4_rope_freqs_params": abi.RopeFreqsParams, "dsv4_rope_params": abi.RopeParams,
               "dsv4_rope_table_params": abi.RopeTableParams, "dsv4_plan_cache": abi.PlanCache,
               "dsv4_batch_plan_params": abi.BatchPlanParams, "dsv4_draft_verify_params": abi.DraftVerifyParams}
    consts = {"DSV4_PLAN_MAX_CACHES": abi.PLAN_MAX_CACHES, "DSV4_PLAN_MAX_REQUESTS": abi.PLAN_MAX_REQUESTS,
              "DSV4_PLAN_MAX_TOKENS": abi.PLAN_MAX_TOKENS}
    consts.update({f"DSV4_ROPE_{k.upper()}": v for k, v in abi.ROPE_SCALINGS.items()})
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', 'int main(void){']
    lines += [f'printf("{k} %d\\n", {k});' for k in consts]
    for cname, st in structs.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in st._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(exe)], check=True)
    got = dict(l.rsplit(" ", 1) for l in subprocess.run([str(exe)], capture_output=True, text=True,
                                                          check=True).stdout.split("\n") if l)
    for k, v in consts.items():
        assert int(got[k]) == v, k
    for cname, st in structs.items():
        assert int(got[cname]) == C.sizeof(st)
        for f, _ in st._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(st, f).offset, (cname, f)


def refused(abi, call, params, status=-1):  # noqa: F811
    """(each is refused before anything is launched: the addresses are never touched)"""
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert getattr(lib, call)(params, None) == status
    assert lib.dsv4_kernel_launches() == n0


# ------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------
def rope_params(abi, **kw):  # noqa: F811
    f = dict(x=0x10000, y=0x20000, x_token_stride=1024, x_head_stride=128, y_token_stride=1024, y_head_stride=128,
             heads=8, heads2=2, dtype=abi.BF16, T=3, head_dim=128, positions=0x30000, freqs=0x40000, rope_dim=64,
             x2_token_stride=256, x2_head_stride=128, y2_token_stride=256, y2_head_stride=128, scale=1.0)
    f.update(kw)
    return abi.make(abi.RopeParams, **f)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(x=0x10008), -1), (dict(y=0x20004), -1), (dict(positions=None), -1),
    (dict(positions=0x30002), -1), (dict(freqs=None), -1), (dict(freqs=0x40008), -1), (dict(dtype=2), -2),
    (dict(T=-1), -1), (dict(T=(1 << 30) + 1), -1), (dict(heads=0), -1), (dict(heads=1025), -1), (dict(head_dim=100), -1),
    (dict(head_dim=8, rope_dim=16), -1), (dict(head_dim=1032), -1), (dict(rope_dim=24), -1), (dict(rope_dim=0), -1),
    (dict(rope_dim=144), -1), (dict(rope_first=72), -1), (dict(rope_first=-8), -1), (dict(rope_first=4), -1),
    (dict(rope_first=2147483640, rope_dim=16), -1), (dict(rope_dim=2147483632), -1), (dict(rope_halves=2), -1),
    (dict(inverse=-1), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(x_token_stride=1020), -1),
    (dict(x_head_stride=-128), -1), (dict(y_token_stride=0), -1), (dict(y_head_stride=0), -1),
    (dict(y=0x10000, y_token_stride=2048), -1), (dict(x2=0x50000), -1), (dict(y2=0x50000), -1),
    (dict(x2=0x50000, y2=0x60000, heads2=0), -1), (dict(x2=0x50000, y2=0x60004), -1), (dict(x2=0x50000, y2=0x20000), -1),
    (dict(x2=0x50000, y2=0x60000, y2_head_stride=0), -1), (dict(struct_size=8), -1),
])
def test_rope_refusals(abi, kw, status):  # noqa: F811
    refused(abi, "dsv4_rope", rope_params(abi, **kw), status)


@pytest.mark.parametrize("kw", [dict(table=None), dict(table=0x10008), dict(freqs=None), dict(freqs=0x20004), dict(rows=-1),
                                dict(rope_dim=12), dict(rope_dim=0), dict(rope_dim=1032), dict(first_position=-1),
                                dict(first_position=2 ** 31 - 3), dict(scale=math.nan), dict(struct_size=4)])
def test_rope_table_refusals(abi, kw):  # noqa: F811
    f = dict(table=0x10000, freqs=0x20000, rows=4, rope_dim=64, scale=1.0)
    f.update(kw)
    refused(abi, "dsv4_rope_table", abi.make(abi.RopeTableParams, **f))


def plan_params(abi, cache=None, **kw):  # noqa: F811
    k = dict(page_size=64, ratio=1, max_pages_per_seq=8, num_pages=100, block_table=0x1000, held=0x2000, held_out=0x2000,
             free_pages=0x3000, free_count=0x4000, free_count_out=0x4000, slots=0x5000)
    k.update(cache or {})
    f = dict(B=4, T=16, num_caches=1, ctx=0x6000, n_new=0x7000, q_start=0x8000, kv_len=0x9000, positions=0xA000)
    f.update(kw)
    p = abi.make(abi.BatchPlanParams, **f)
    p.caches[0] = abi.PlanCache(**k)
    return p


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=4097), dict(T=-1), dict(T=(1 << 19) + 1), dict(num_caches=0), dict(num_caches=5),
    dict(num_caches=2), dict(ctx=None), dict(n_new=None), dict(q_start=None), dict(kv_len=None), dict(ctx=0x6002),
    dict(ctx_add=0x6001), dict(ctx_out=0x6003), dict(positions=0xA004), dict(token_seq=0xA008), dict(struct_size=8),
    dict(cache=dict(page_size=0)), dict(cache=dict(page_size=65537)), dict(cache=dict(ratio=0)),
    dict(cache=dict(ratio=65537)), dict(cache=dict(window=-1)), dict(cache=dict(window=8)),
    dict(cache=dict(window=8, ratio=4, first=0x100, first_out=0x100)), dict(cache=dict(first=0x100, first_out=0x100)),
    dict(cache=dict(window=8, first=0x100)), dict(cache=dict(max_pages_per_seq=0)),
    dict(cache=dict(max_pages_per_seq=(1 << 19) + 1)), dict(cache=dict(num_pages=-1)), dict(cache=dict(num_pages=1 << 31)),
    dict(cache=dict(block_table=None)), dict(cache=dict(held=None)), dict(cache=dict(held_out=None)),
    dict(cache=dict(free_pages=None)), dict(cache=dict(free_count=None)), dict(cache=dict(free_count_out=None)),
    dict(cache=dict(slots=0x5008)), dict(cache=dict(free_pages=0x3002)),
])
def test_plan_refusals(abi, kw):  # noqa: F811
    refused(abi, "dsv4_batch_plan", plan_params(abi, **kw))


@pytest.mark.parametrize("shared", ["block_table", "held_out", "free_pages", "free_count_out", "slots", "first_out"])
def test_plan_refuses_caches_that_share_what_they_write(abi, shared):  # noqa: F811
    a = dict(page_size=64, ratio=1, window=8, max_pages_per_seq=8, num_pages=100, block_table=0x1000, held=0x2000,
             held_out=0x2100, first=0x2200, first_out=0x2300, free_pages=0x3000, free_count=0x4000, free_count_out=0x4100,
             slots=0x5000)
    b = {k: v + 0x100000 if v >= 0x1000 else v for k, v in a.items()}
    p = plan_params(abi, cache=a, num_caches=2)
    p.caches[1] = abi.PlanCache(**dict(b, **{shared: a[shared]}))
    refused(abi, "dsv4_batch_plan", p)


def verify_params(abi, **kw):  # noqa: F811
    f = dict(target=0x10000, target_stride=100, target_dtype=abi.BF16, tokens=0x2000, q_start=0x3000, T=8, B=2, vocab=100,
             max_q_len=4, u=0x4000, noise=0x5000, noise_stride=100, out_tokens=0x6000, n_out=0x7000, draft_dtype=abi.BF16,
             draft_stride=100, draft_rows=6)
    f.update(kw)
    return abi.make(abi.DraftVerifyParams, **f)


@pytest.mark.parametrize("kw,status", [
    (dict(target=None), -1), (dict(target=0x10001), -1), (dict(target_dtype=2), -2),
    (dict(target_dtype=0, target=0x10002), -1), (dict(target_stride=99), -1), (dict(target_probs=2), -1),
    (dict(tokens=None), -1), (dict(tokens=0x2002), -1), (dict(q_start=None), -1), (dict(T=-1), -1), (dict(B=-1), -1),
    (dict(B=65536), -1), (dict(T=(1 << 30) + 1), -1), (dict(vocab=0), -1), (dict(vocab=(1 << 24) + 1), -1),
    (dict(max_q_len=0), -1), (dict(u=None), -1), (dict(noise=None), -1), (dict(noise_stride=99), -1),
    (dict(noise=0x5002), -1), (dict(u=0x4001), -1), (dict(out_tokens=None), -1), (dict(n_out=None), -1),
    (dict(logp=0x6002), -1), (dict(temperature=0x6002), -1), (dict(draft=0x20000, draft_stride=50), -1),
    (dict(draft=0x20001), -1), (dict(draft=0x20000, draft_rows=-1), -1), (dict(draft=0x20000, draft_dtype=3), -2),
    (dict(draft_probs=-1), -1), (dict(draft_row=0x6001), -1), (dict(struct_size=0), -1),
])
def test_verify_refusals(abi, kw, status):  # noqa: F811
    refused(abi, "dsv4_draft_verify", verify_params(abi, **kw), status)


def test_empty_calls_pass(abi):  # noqa: F811
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert lib.dsv4_rope(rope_params(abi, T=0, x=None, positions=None), None) == 0
    assert lib.dsv4_rope_table(abi.make(abi.RopeTableParams, rope_dim=64, scale=1.0), None) == 0
    assert lib.dsv4_draft_verify(verify_params(abi, B=0, q_start=None), None) == 0
    assert lib.dsv4_kernel_launches() == n0


def test_python_binding_refuses():
    import deepseek_v4_hybrid_gb300 as M
    x = torch.zeros((2, 3, 32))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        M.rope_params(x, x, i, torch.zeros(16, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        M.rope_table_params(torch.zeros((4, 32)), torch.zeros(16, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        M.plan_cache(torch.zeros((2, 3), dtype=torch.int32), i, i, i[:1], 16)
    with pytest.raises(ValueError, match="CUDA"):
        M.batch_plan_params(i, i, i, i, [])
    with pytest.raises(ValueError, match="CUDA"):
        M.draft_verify_params(x[0], i, i, 1, i, i)
    with pytest.raises(ValueError, match="none of"):
        M.rope_freqs(64, scaling="twice", device="cpu")


# ------------------------------------------------------------------------------------------------
# frequencies
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [2, 16, 64, 128, 1024])
@pytest.mark.parametrize("kw", [dict(), dict(theta=500000.0), dict(scaling="linear", factor=4.0),
                                dict(scaling="base", factor=8.0), dict(scaling="yarn", factor=40.0, original_len=4096),
                                dict(scaling="yarn", factor=2.0, original_len=3, beta_fast=32, beta_slow=1),
                                dict(scaling="bands", factor=8.0, original_len=8192),
                                dict(scaling="bands", factor=8.0, original_len=100, low_turns=0.5, high_turns=9.0)],
                         ids=lambda k: "_".join(f"{v}" for v in k.values()) or "plain")
def test_frequencies(dim, kw):
    """Against the formulas in Python's float64: each is a power (some 30 ulp at exponents up to 2^5) and a few roundings,
    the fraction is cut below 2^-64."""
    import deepseek_v4_hybrid_gb300 as M
    if kw.get("scaling") == "base" and dim == 2:
        with pytest.raises(M.Dsv4Error):
            M.rope_freqs(dim, device="cpu", **kw)
        return
    got = M.rope_freqs(dim, device="cpu", **kw).numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64
    want = L.frequencies(dim, **kw) / (2 * math.pi)
    assert got[0] <= 1 / (2 * math.pi) * (1 + 2 ** -50)
    np.testing.assert_allclose(got, want, rtol=2 ** -46, atol=2.0 ** -63)


@pytest.mark.parametrize("kw", [dict(dim=3), dict(theta=1.0), dict(theta=math.inf), dict(factor=0.5), dict(factor=math.nan),
                                dict(scaling="yarn"), dict(scaling="yarn", original_len=4096, beta_fast=0.0),
                                dict(scaling="bands"), dict(scaling="bands", original_len=64, low_turns=4.0),
                                dict(scaling="base", factor=1e300, dim=4), dict(dim=1026)])
def test_frequencies_refused(kw):
    import deepseek_v4_hybrid_gb300 as M
    kw = dict(kw)
    with pytest.raises((M.Dsv4Error, ValueError)):
        M.rope_freqs(kw.pop("dim", 64), device="cpu", **kw)


# ------------------------------------------------------------------------------------------------
# the oracle's own pins
# ------------------------------------------------------------------------------------------------
def test_oracle_angles_of_far_positions():
    """The reduced angle against a product in Python's integers and fractions, up to 2^31 - 1."""
    from fractions import Fraction
    f = np.array([0x28BE60DB9391054A, 12345678901234567, 1], np.uint64)
    pos = np.array([0, 1, 7, 4095, 1 << 20, 2 ** 31 - 1])
    w = L.angles(pos, f)
    for i, p in enumerate(pos):
        for j in range(3):
            turns = Fraction(int(p) * int(f[j]) % 2 ** 64, 2 ** 64)
            turns = turns - 1 if turns >= Fraction(1, 2) else turns
            assert abs(w[i, j] - float(turns) * 2 * math.pi) <= 2 ** -50


def test_oracle_rotation():
    """Lengths stay, q . k depends on the distance, the inverse turns back, and the inverse is the transpose (the
    gradient of the forward turn)."""
    g = np.random.default_rng(0)
    f = np.round(L.frequencies(16) / (2 * math.pi) * 2.0 ** 64).astype(np.uint64)
    q, k = g.standard_normal((2, 1, 1, 24))
    for halves in (False, True):
        turn = lambda x, p, **kw: L.rope(x, [p], f, first=8, halves=halves, **kw)  # noqa: E731
        assert abs(np.linalg.norm(turn(q, 90)) - np.linalg.norm(q)) < 1e-12
        assert abs((turn(q, 90) * turn(k, 71)).sum() - (turn(q, 1019) * turn(k, 1000)).sum()) < 1e-11
        np.testing.assert_allclose(turn(turn(q, 55), 55, inverse=True), q, atol=1e-14)
        assert abs((turn(q, 55, scale=1.5) * k).sum() - (q * turn(k, 55, scale=1.5, inverse=True)).sum()) < 1e-13
        eps, at = 1e-6, 11  # against differences
        step = np.zeros_like(q)
        step[..., at] = eps
        slope = ((turn(q + step, 55) - turn(q - step, 55)) * k).sum() / (2 * eps)
        assert abs(slope - turn(k, 55, inverse=True)[0, 0, at]) < 1e-8


def test_oracle_plan_by_hand():
    """Pages of 4 rows.  Request 0 kept 6 rows of 12 and brings 1: its third page goes back and is the first
    one taken again, by request 1 (full pages, one more row); request 2 has ended; request 3 begins with 9 rows and finds
    two pages of three."""
    table = np.array([[0, 1, 2, -1], [3, 4, -1, -1], [5, -1, -1, -1], [-1, -1, -1, -1]])
    k = L.Cache(4, 1, 0, table, np.array([3, 2, 1, 0]), np.zeros(4, int), np.array([9, -1, -1, -1]), 1)
    k.stack = np.concatenate([k.stack, np.full(8, -1)])
    r = L.plan([6, 8, 0, 0], [0, 0, 0, 0], [1, 1, 0, 9], 16, [k])
    # stack after what is given back: 9, 2 (request 0), 5 (request 2); popped: 5 for request 1; 3 pages do not fit
    assert list(k.held) == [2, 3, 0, 0] and k.table[1, 2] == 5 and k.count == 2 and list(k.stack[:3]) == [9, 2, 5]
    assert list(r["q_start"]) == [0, 1, 2, 2, 2] and list(r["kv_len"]) == [7, 9, 0, 0]
    assert list(r["positions"][:3]) == [6, 8, -1] and list(r["slots"][0][:3]) == [1 * 4 + 2, 5 * 4, -1]
    assert not r["flagged"]


def test_oracle_verify_keeps_the_targets_distribution():
    """Drawn from q and verified, tokens follow p: 40,000 draws over five tokens, each frequency within five standard
    deviations."""
    g = np.random.default_rng(1)
    p, q = np.array([0.4, 0.3, 0.2, 0.1, 0.0]), np.array([0.1, 0.2, 0.3, 0.2, 0.2])
    N = 40000
    drawn = g.choice(5, N, p=q)
    tokens = np.stack([np.zeros(N, int), drawn], 1).ravel()
    start = np.arange(N + 1) * 2
    target = np.tile(np.log(np.maximum(p, 1e-300)), (2 * N, 1))
    out, count, _, _ = L.verify(target, tokens, start, 2, draft=np.tile(q, (N, 1)), draft_probs=True,
                                u=g.random(2 * N), noise=g.exponential(size=(N, 5)))
    freq = np.bincount(out[:, 0], minlength=5) / N
    assert np.all(np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / N) + 1e-12)
    assert abs((count == 2).mean() - np.minimum(p, q).sum()) < 5 * 0.5 / math.sqrt(N)
