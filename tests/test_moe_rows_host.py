"""The tile-width override of the mixture-of-experts layer: host state, no GPU needed."""
import pytest

import linear_algebra_sgemm_amd as lib


@pytest.mark.parametrize("rows", [16, 32, 64, 0])
def test_force_moe_rows_accepts(rows):
    assert lib.gemm_debug_force_moe_rows(rows) == lib.STATUS_SUCCESS


@pytest.mark.parametrize("rows", [-1, 1, 8, 48, 128])
def test_force_moe_rows_refuses(rows):
    assert lib.gemm_debug_force_moe_rows(rows) == lib.STATUS_INVALID_VALUE
