"""Limits of the grouped plans that no GPU test can reach: sizes whose 32-bit arithmetic on the device
would wrap are refused when the plan is made."""
import pytest

import tiled_gemm_epilogues_amd as tge

LIM31 = 1 << 31


@pytest.mark.parametrize("ab,cd", [("f16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_gradient_rows_leave_room_for_a_step(ab, cd):
    # the kernels step over the rows of a range up to 256 at a time, in 32 bits: a range that ends
    # less than a step below 2^31 would wrap, and the bias sums would then read in front of B
    for rows, status in ((LIM31 - 1, tge.STATUS_NOT_SUPPORTED), (LIM31 - 1023, tge.STATUS_NOT_SUPPORTED),
                         (LIM31 - 1024, tge.STATUS_SUCCESS)):
        st, h = tge.gemm_grouped_grad_plan_create(rows, 8, 8, 2, 8, 8, 8, 64, ab, cd)
        assert st == status, rows
        tge.gemm_grouped_plan_destroy(h)


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("algo,tile", [("auto", 0), ("fast", 256), ("staged", 128), ("skinny", 0), ("general", 128)])
def test_rows_are_bounded_by_the_grid(algo, tile, op_b):
    # rows plans step by their tile: 2^23 workgroups of at most 128 rows stay below 2^30
    for ab in ("f16", "f32"):
        st, h = tge.gemm_grouped_plan_create(1 << 30, 64, 64, 1, op_b, 64, 64, 64, 4096, 64, ab, ab, "none", algo, tile)
        assert st == tge.STATUS_NOT_SUPPORTED and h is None
