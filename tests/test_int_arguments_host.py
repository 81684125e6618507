"""Whole numbers past 32 bits do not reach the C ABI as their low bits."""
from group_wise_affine_qmv_b200 import aq


def test_int32_saturates():
    for v in (0, 5, -1, 2 ** 31 - 1, -2 ** 31):
        assert aq._int32(v) == v
    assert aq._int32(2 ** 32 + 5) == aq._int32(2 ** 63) == 2 ** 31 - 1
    assert aq._int32(-2 ** 32 + 5) == -2 ** 31
