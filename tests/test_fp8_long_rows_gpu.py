"""GPU test of the block-scaled product at the longest rows there are: 2^31 - 1 columns, on the tile of
the rule and on tiles whose column numbers end before that."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_fp8_gpu import E4M3, library  # noqa: F401  (the library's lifetime)

pytestmark = pytest.mark.gpu


def test_longest_rows():
    K = 2 ** 31 - 1
    one = torch.tensor([1.0]).to(E4M3).view(torch.uint8).item()
    A = torch.zeros(K, dtype=torch.uint8, device="cuda")
    A[::1 << 20] = one                    # 2048 ones, and the last column
    A[K - 1] = one
    S = torch.ones(-(-K // 128), device="cuda")
    C = torch.empty(1, device="cuda")
    for tile in (-1, 1, 4):
        note("fp8 longest rows tile %d" % tile)
        assert lib.gemm_debug_force_tile(2, tile) == lib.STATUS_SUCCESS
        try:
            C.fill_(-1)
            lib.fp8_gemm_bias_act(1, 1, K, 1.0, A, K, S, 1, A, K, S, 1, 128, None, lib.ACT_NONE,
                                  lib.TYPE_F32, C, 1)
            torch.cuda.synchronize()
        finally:
            lib.gemm_debug_force_tile(2, -1)
        assert C.item() == 2049
