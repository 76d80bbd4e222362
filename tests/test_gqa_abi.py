"""The grouped-query calls of the C ABI: symbols, struct layouts and refusals, without a GPU; and the
oracle's own pins."""
import ctypes as C
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import dsv4_oracle as O
from oracle import gqa_oracle as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dsv4_gqa.h")


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    lib_path = os.path.join(ROOT, "deepseek_v4_hybrid_gb300", "_lib", "libdsv4.so")
    if not os.path.exists(lib_path):
        __graft_entry__._build_module().build()
    from deepseek_v4_hybrid_gb300 import _abi
    _abi.load()
    return _abi


def test_exports_and_struct_layout(abi, tmp_path):
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(dsv4_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(abi.GQA_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", abi.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\bT (dsv4_\w+)", out))
    structs = {"dsv4_gqa_append_params": abi.GqaAppendParams, "dsv4_gqa_attention_params": abi.GqaAttentionParams}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', 'int main(void){',
             'printf("e4m3 %d\\n", DSV4_E4M3_PAGE);']
    for cname, st in structs.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in st._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(exe)], check=True)
    got = dict(l.rsplit(" ", 1) for l in subprocess.run([str(exe)], capture_output=True, text=True,
                                                          check=True).stdout.split("\n") if l)
    assert int(got["e4m3"]) == abi.E4M3_PAGE
    for cname, st in structs.items():
        assert int(got[cname]) == C.sizeof(st)
        for f, _ in st._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(st, f).offset, (cname, f)


def append_params(abi, **kw):
    f = dict(T=2, B=1, q_heads=8, kv_heads=2, head_dim=128, page_size=64, num_pages=4, max_pages_per_seq=2, max_q_len=2,
             cache_dtype=abi.E4M3_PAGE, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128,
             k_page_stride=16384, k_cache_head_stride=8192, k_row_stride=128, v_page_stride=16384,
             v_cache_head_stride=8192, v_row_stride=128, q_token_stride=1024, q_head_stride=128, q_out_token_stride=1024,
             q_out_head_stride=128, rope_dim=64, max_pos=100)
    for name in ("k_new", "v_new", "k_cache", "v_cache", "k_exp", "v_exp", "block_table", "q_start", "kv_len"):
        f[name] = 0x10000
    f.update(kw)
    return abi.make(abi.GqaAppendParams, **f)


# (each is refused before anything is launched: the addresses are never touched)
@pytest.mark.parametrize("kw,status", [
    (dict(k_new=None), -1), (dict(v_new=0x10008), -1), (dict(k_cache=None), -1), (dict(v_cache=0x10004), -1),
    (dict(k_exp=None), -1), (dict(block_table=None), -1), (dict(q_start=0x10002), -1), (dict(kv_len=None), -1),
    (dict(head_dim=96), -2), (dict(page_size=48), -2), (dict(page_size=0), -2), (dict(cache_dtype=2), -2),
    (dict(max_q_len=0), -1), (dict(T=-1), -1), (dict(B=-1), -1), (dict(B=70000), -1), (dict(kv_heads=0), -1),
    (dict(q_heads=2000), -1), (dict(num_pages=-1), -1), (dict(num_pages=1 << 31), -1), (dict(max_pages_per_seq=0), -1),
    (dict(k_token_stride=4), -1), (dict(k_row_stride=64), -1), (dict(v_row_stride=136), -1), (dict(k_page_stride=0), -1),
    (dict(v_cache_head_stride=-8192), -1),
    (dict(q=0x20000), -1), (dict(q=0x20000, q_out=0x30004), -1), (dict(q=0x20000, q_out=0x20000, q_out_token_stride=2048), -1),
    (dict(cos_sin=0x20000, rope_dim=24), -1), (dict(cos_sin=0x20000, rope_first=4), -1),
    (dict(cos_sin=0x20000, rope_first=72), -1), (dict(cos_sin=0x20000, max_pos=0), -1), (dict(cos_sin=0x20008), -1),
    (dict(struct_size=8), -1),
])
def test_append_refusals(abi, kw, status):
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert lib.dsv4_gqa_append(append_params(abi, **kw), None) == status
    assert lib.dsv4_kernel_launches() == n0


def attention_params(abi, **kw):
    f = dict(T=2, B=1, q_heads=8, kv_heads=2, head_dim=128, page_size=64, num_pages=4, max_pages_per_seq=2, max_q_len=2,
             cache_dtype=abi.E4M3_PAGE, k_page_stride=16384, k_cache_head_stride=8192, k_row_stride=128,
             v_page_stride=16384, v_cache_head_stride=8192, v_row_stride=128, q_token_stride=1024, q_head_stride=128,
             max_kv_len=100, softmax_scale=0.1, causal=1, out_dtype=abi.BF16, workspace_bytes=1 << 40)
    for name in ("q", "out", "k_cache", "v_cache", "k_exp", "v_exp", "block_table", "q_start", "kv_len", "workspace"):
        f[name] = 0x10000
    f.update(kw)
    return abi.make(abi.GqaAttentionParams, **f)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(q=0x10008), -1), (dict(out=None), -1), (dict(out=0x10004), -1), (dict(k_cache=0x10008), -1),
    (dict(v_exp=None), -1), (dict(q_heads=7), -1), (dict(head_dim=256), -2), (dict(page_size=8), -2),
    (dict(page_size=512), -2), (dict(out_dtype=2), -2), (dict(cache_dtype=0), -2), (dict(max_kv_len=-1), -1),
    (dict(max_kv_len=(1 << 30) + 1), -1), (dict(window=-1), -1), (dict(causal=2), -1), (dict(softcap=-1.0), -1),
    (dict(softcap=math.inf), -1), (dict(softmax_scale=math.nan), -1), (dict(q_token_stride=1023), -1),
    (dict(workspace=None), -1), (dict(workspace=0x10080), -1), (dict(workspace_bytes=0), -1), (dict(lse=0x10001), -1),
    (dict(kv_start=0x10002), -1), (dict(sink=0x10002), -1), (dict(struct_size=8), -1), (dict(max_q_len=0), -1),
])
def test_attention_refusals(abi, kw, status):
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert lib.dsv4_gqa_attention(attention_params(abi, **kw), None) == status
    assert lib.dsv4_kernel_launches() == n0


@pytest.mark.parametrize("kw", [dict(softcap=2000.0), dict(softcap=1e-39, softmax_scale=8.0), dict(T=(1 << 30) + 1)])
def test_attention_refuses_caps_and_counts_out_of_range(abi, kw):
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert lib.dsv4_gqa_attention(attention_params(abi, **kw), None) == -1
    assert lib.dsv4_gqa_attention_workspace_bytes(attention_params(abi, **kw)) == 0
    assert lib.dsv4_kernel_launches() == n0


@pytest.mark.parametrize("kw", [dict(q_out_token_stride=0), dict(q_out_head_stride=0)])
def test_append_refuses_queries_written_over_one_another(abi, kw):
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert lib.dsv4_gqa_append(append_params(abi, q=0x20000, q_out=0x30000, **kw), None) == -1
    assert lib.dsv4_gqa_append(append_params(abi, T=(1 << 30) + 1), None) == -1
    assert lib.dsv4_kernel_launches() == n0


def test_workspace_is_zero_for_refused_params_and_empty_calls_pass(abi):
    lib = abi.load()
    assert lib.dsv4_gqa_attention_workspace_bytes(attention_params(abi)) > 0
    assert lib.dsv4_gqa_attention_workspace_bytes(attention_params(abi, head_dim=96)) == 0
    assert lib.dsv4_gqa_attention(attention_params(abi, T=0, q=None, workspace=None), None) == 0
    assert lib.dsv4_gqa_append(append_params(abi, T=0, k_new=None), None) == 0
    assert lib.dsv4_gqa_append(append_params(abi, B=0, k_cache=None), None) == 0


def test_python_binding_refuses_host_tensors():
    import __graft_entry__  # noqa: F401
    import deepseek_v4_hybrid_gb300 as M
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        M.gqa_append_params(k, k, cache, cache, i[None, :1], i, i[:1], 1)


# ------------------------------------------------------------------------------------------------
# the oracle's own pins
# ------------------------------------------------------------------------------------------------
def test_oracle_rotation_keeps_lengths_and_relative_angles():
    """With a true cos/sin table, rotating q at p and k at j leaves lengths, and q.k depends on p - j only."""
    g = np.random.default_rng(0)
    half = 16
    ang = np.arange(50)[:, None] * 10.0 ** (-np.arange(half) / half)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    q, k = g.standard_normal((2, 64)).astype(np.float32)
    for halves in (False, True):
        r = lambda x, p: G.rotate(x, p, cs, 8, halves).astype(np.float64)  # noqa: E731
        assert abs(np.linalg.norm(r(q, 30)) - np.linalg.norm(q)) < 1e-5
        assert abs(r(q, 30) @ r(k, 23) - r(q, 17) @ r(k, 10)) < 1e-4
        np.testing.assert_array_equal(r(q, 0), q)
        np.testing.assert_array_equal(r(q, 9)[:8], q[:8])


def test_oracle_append_growth_by_hand():
    """One page, one head: a row of maximum 448 (exponent 0), then one of 3584 = 448 * 8 (exponent 3): the first
    row's codes lose 3 binary exponents, small ones rounding to even among the subnormals."""
    cache, exp = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.uint8)
    k = np.zeros((1, 1, 64), np.float32)
    k[0, 0, :4] = (448, 1, 2 ** -6, 3 * 2 ** -9)
    z = np.zeros_like(k)
    c2, e2 = cache.copy(), exp.copy()
    G.append(k, z, [cache, c2], [exp, e2], np.zeros((1, 1), int), np.array([0, 1]), np.array([1]))
    assert exp[0, 0] == 127 and e2[0, 0] == 0
    assert list(O.e4m3_decode(cache[0, 0, 0, :4])) == [448, 1, 2 ** -6, 3 * 2 ** -9]
    G.append(k * 8, z, [cache, c2], [exp, e2], np.zeros((1, 1), int), np.array([0, 1]), np.array([2]))
    assert exp[0, 0] == 130
    assert list(O.e4m3_decode(cache[0, 0, 0, :4])) == [56, 0.125, 2 ** -9, 0]
    assert list(O.e4m3_decode(cache[0, 0, 1, :4])) == [448, 1, 2 ** -6, 3 * 2 ** -9]


def test_oracle_attention_against_dense_softmax():
    from gqa_cases import Batch
    bt = Batch([5, 1], [20, 33], 4, 2, 64, 16, "bf16", seed=4)
    out, lse, _, _ = G.attention(bt.q64(), bt.caches, None, bt.table, bt.q_start, bt.kv, 0.3)
    k = O.bf16_decode(bt.caches[0])[bt.table[0, :2], 1].reshape(-1, 64)[:20].astype(np.float64)
    v = O.bf16_decode(bt.caches[1])[bt.table[0, :2], 1].reshape(-1, 64)[:20].astype(np.float64)
    z = torch.from_numpy(bt.q64()[2, 3] @ k[:18].T * 0.3)
    np.testing.assert_allclose(out[2, 3], (torch.softmax(z, 0) @ torch.from_numpy(v[:18])).numpy(), rtol=1e-12,
                               atol=1e-14)  # 18 terms of magnitude O(1): 18 * 2^-53
    np.testing.assert_allclose(lse[2, 3], torch.logsumexp(z, 0).item(), rtol=1e-12)
