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
