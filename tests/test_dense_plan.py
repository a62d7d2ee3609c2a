"""The choice of how a dense product runs, on the host: its refusals, its limits,
and that the sizes of the GPU tests take every way there is."""
import ctypes

import pytest

import dense_shapes
from group_limited_routed_moe_b200 import moe


def test_every_way_is_among_the_tested_sizes():
    assert not dense_shapes.uncovered()


@pytest.mark.parametrize("args", [
    (-1, 4, 64, 64), (6, 4, 64, 64), (0, 0, 64, 64), (0, -1, 64, 64), (0, 4, 12, 64), (0, 4, 64, 12), (5, 4, 0, 64),
    (5, 4, 64, 24), (5, (1 << 22) + 1, 64, 64),
])
def test_refusals(args):
    plan = (ctypes.c_int32 * 4)()
    assert moe.lib.moe_dense_plan(*args, plan) == moe.MOE_ERR_INVALID_ARG
    assert moe.lib.moe_dense_plan(*args[:1], 4, 64, 64, None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("T", [1, 16, 17, 32, 33, 300, 1 << 22])
def test_limits(T):
    """The largest and smallest sizes have a way, inside the kernels' limits."""
    for p in moe.PRODUCTS:
        for N in (8, 4096, 65536):
            for K in (16, 1536, 65536):
                kernel, tile, rows, split = moe.dense_plan(p, T, N, K)
                if kernel == "pairs":
                    assert tile in (128, 256) and rows == 256 and 1 <= split <= 4
                else:
                    assert p != "dw" and tile in (16, 32, 64) and rows in (64, 128) and split in (1, 2, 4, 8)
                    assert p != "gate_up" or rows == 128
