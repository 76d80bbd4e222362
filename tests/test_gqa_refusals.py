"""Refusals of the grouped-query calls whose numbers would leave the types they are computed in; no GPU needed."""
import pytest

from test_gqa_abi import abi, append_params, attention_params  # noqa: F401

INT_MAX = 2 ** 31 - 1


# (each is refused before anything is launched: the addresses are never touched)
@pytest.mark.parametrize("first,dim", [(16, 2147483632), (2147483640, 16), (64, INT_MAX - 15), (0, 2147483632),
                                       (2147483640, 2147483632), (120, 16), (0, 144), (128, 16)])
def test_append_refuses_rotations_beyond_the_head(abi, first, dim):  # noqa: F811
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    assert lib.dsv4_gqa_append(append_params(abi, cos_sin=0x20000, rope_first=first, rope_dim=dim), None) == -1
    assert lib.dsv4_kernel_launches() == n0


@pytest.mark.parametrize("cap,scale", [(1e-39, 1e-30), (1e-39, 0.0), (1e-44, -1e-20), (0.0, 3e38), (0.0, -1e38), (5.0, 2e38)])
def test_attention_refuses_scales_that_leave_fp32(abi, cap, scale):  # noqa: F811
    """2 log2(e) / softcap and log2(e) softmax_scale are fp32 factors: infinite ones turn a score of 0 into NaN."""
    lib, n0 = abi.load(), abi.load().dsv4_kernel_launches()
    p = attention_params(abi, softcap=cap, softmax_scale=scale)
    assert lib.dsv4_gqa_attention(p, None) == -1
    assert lib.dsv4_gqa_attention_workspace_bytes(p) == 0
    assert lib.dsv4_kernel_launches() == n0


@pytest.mark.parametrize("cap,scale", [(2e-38, 1e-3), (1e-3, 8e37 * 1e-3), (0.0, 8e37), (1024.0, -1.0)])
def test_attention_takes_scales_within_fp32(abi, cap, scale):  # noqa: F811
    assert abi.load().dsv4_gqa_attention_workspace_bytes(attention_params(abi, softcap=cap, softmax_scale=scale)) > 0
