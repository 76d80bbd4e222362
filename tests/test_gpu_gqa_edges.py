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


