"""The calls around the layers: what is refused because tensors of one call share memory (CPU: nothing is launched)."""
import itertools

import numpy as np
import pytest
import torch

from test_gqa_abi import abi  # noqa: F401
from test_loop_abi import plan_params, refused, rope_params

BASE = 1 << 20


def rope_call(abi, T, D, x, y, x2=None, y2=None, dtype=None):  # noqa: F811
    """Each of x, y, x2, y2 as (first element, token stride, head stride, heads)."""
    dtype = abi.BF16 if dtype is None else dtype
    size = 4 if dtype == abi.F32 else 2
    f = dict(dtype=dtype, T=T, head_dim=D, rope_dim=16, heads=x[3], heads2=1)
    for name, t in (("x", x), ("y", y), ("x2", x2), ("y2", y2)):
        if t is not None:
            f.update({name: BASE + size * t[0], f"{name}_token_stride": t[1], f"{name}_head_stride": t[2]})
    if x2 is not None:
        f["heads2"] = x2[3]
    return rope_params(abi, **f)


Q, K = (0, 640, 64, 4), (256, 640, 64, 2)         # of a fused projection of 10 heads of 64
FAR, FAR2 = (100000, 256, 64, 4), (200000, 128, 64, 2)


@pytest.mark.parametrize("x,y,x2,y2", [
    (Q, (8, 640, 64, 4), None, None), (Q, (64, 640, 64, 4), None, None),
    (Q, (640, 640, 64, 4), None, None), (Q, (640 * 2 + 192, 640, 64, 4), None, None),
    (Q, (0, 256, 64, 4), None, None), ((0, 0, 64, 4), (0, 256, 64, 4), None, None),
    (Q, FAR, K, Q[:3] + (2,)), (Q, K[:3] + (4,), K, FAR2), (Q, FAR, K, FAR[:3] + (2,)), (Q, Q, K, (192, 640, 64, 2)),
    (Q, FAR, K, (100000 + 56, 256, 64, 2)), (Q, Q, K, (640 - 64, 640, 64, 2)),
    ((0, 64, 1024, 4), (64 * 20, 64, 1024, 4), None, None),                       # heads outside tokens, 30 tokens
    ((0, 128, 64, 1), (32, 128, 64, 1), None, None),
    ((0, 256, 64, 4), (100000, 56, 64, 4), None, None), ((0, 256, 64, 4), (100000, 256, 56, 4), None, None),
    ((0, 256, 64, 4), (100000, 64, 64, 4), None, None),                           # rows of y over one another
])
def test_rope_refuses_rows_that_meet(abi, x, y, x2, y2):  # noqa: F811
    refused(abi, "dsv4_rope", rope_call(abi, 30, 64, x, y, x2, y2))


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the check would be launched")
def test_rope_rows_of_y_lie_apart(abi):  # noqa: F811
    """Any strides of y: refused exactly where two of its rows share an element."""
    g = np.random.default_rng(1)
    lib, seen = abi.load(), [0, 0]
    for _ in range(6000):
        T, heads, D = int(g.integers(1, 7)), int(g.integers(1, 6)), 16
        token, head = 8 * int(g.integers(2, 14)), 8 * int(g.integers(2, 14))
        at = sorted(t * token + h * head for t, h in itertools.product(range(T), range(heads)))
        meet = any(b - a < D for a, b in zip(at, at[1:]))
        status = lib.dsv4_rope(rope_call(abi, T, D, (0, 1024, 64, heads), (10 ** 6, token, head, heads)), None)
        assert status == (-1 if meet else -3), (T, heads, token, head)
        seen[meet] += 1
    assert min(seen) > 500


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the check would be launched")
def test_rope_row_check_against_every_row(abi):  # noqa: F811
    """Parts of one buffer are refused exactly where two rows meet: every pair of rows compared.  A call that passes the
    check ends at the launch, for want of a device."""
    g = np.random.default_rng(0)
    lib, seen = abi.load(), [0, 0]
    for _ in range(6000):
        T, D, nx, ny = int(g.integers(1, 5)), 16, int(g.integers(1, 4)), int(g.integers(1, 4))
        head, token, off = 8 * int(g.integers(2, 8)), 8 * int(g.integers(2, 30)), 8 * int(g.integers(-40, 41))
        wide, narrow, count = max(token, head), min(token, head), max(nx, ny) if token >= head else T
        if wide < narrow * (count - 1) + D and T > 1:
            continue  # (rows laid through one another otherwise than one stride inside the other)
        rows = lambda at, n: [at + t * token + h * head for t, h in itertools.product(range(T), range(n))]  # noqa: E731
        meet = any(abs(p - q) < D for p in rows(1000, nx) for q in rows(1000 + off, ny))
        x, y2 = (1000, token, head, nx), (1000 + off, token, head, ny)
        status = lib.dsv4_rope(rope_call(abi, T, D, x, (10 ** 6, 256, 64, nx), (2 * 10 ** 6, 256, 64, ny), y2), None)
        assert status == (-1 if meet else -3), (T, nx, ny, head, token, off)
        seen[meet] += 1
    assert min(seen) > 500


@pytest.mark.parametrize("in_place", [True, False], ids=["in place", "apart"])
@pytest.mark.parametrize("order", [(0, 1), (1, 0)], ids=["first writes", "second writes"])
@pytest.mark.parametrize("name", ["held", "first", "free_count"])
def test_plan_refuses_caches_that_read_what_another_writes(abi, name, order, in_place):  # noqa: F811
    """The numbers that one cache advances are the other's input (which is then read behind the store)."""
    caches = []
    for i in range(2):
        at = 0x100000 * (i + 1)
        caches.append(dict(page_size=64, ratio=1, window=8, max_pages_per_seq=8, num_pages=100, block_table=at + 0x1000,
                           held=at + 0x2000, held_out=at + 0x2100, first=at + 0x2200, first_out=at + 0x2300,
                           free_pages=at + 0x3000, free_count=at + 0x4000, free_count_out=at + 0x4100, slots=at + 0x5000))
    writer, reader = caches[order[0]], caches[order[1]]
    reader[name] = writer[name + "_out"]
    if in_place:
        writer[name] = writer[name + "_out"]
    p = plan_params(abi, cache=caches[0], num_caches=2)
    p.caches[1] = abi.PlanCache(**caches[1])
    refused(abi, "dsv4_batch_plan", p)
