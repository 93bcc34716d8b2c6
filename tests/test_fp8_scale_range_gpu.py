"""GPU tests of the block-scaled product with scales far from 1.  The bound is test_fp8_gpu.py's
for exact sums, (128 + blocks + 16) 2^-24 of sum |s_a a s_b b| (fast sums: 2^-11 more), and 2^-125
for every block whose scales' product is below 2^-126."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_fp8_gpu import U, blocks, library, operands  # noqa: F401

pytestmark = pytest.mark.gpu

M, N, K = 130, 260, 520


def product(a, sa, b, sb, b_rows, tile, fast):
    C = torch.empty((M, N), device="cuda")
    assert lib.gemm_debug_force_tile(2, tile) == lib.STATUS_SUCCESS
    try:
        lib.fp8_gemm_bias_act(M, N, K, 1.0, a.view(torch.uint8).cuda(), K, sa.cuda(), M,
                              b.view(torch.uint8).cuda(), K, sb.cuda(), sb.shape[1], b_rows, None,
                              lib.ACT_NONE, lib.TYPE_F32, C, N, fast_sums=fast)
        torch.cuda.synchronize()
    finally:
        lib.gemm_debug_force_tile(2, -1)
    return C.cpu().double()


def wide(q, s, b_rows):
    f = s.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * f.repeat_interleave(b_rows, 0)[:q.shape[0]]


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("tile", range(-1, 11))
def test_far_scales(tile, b_rows, fast):
    a, sa, b, sb = operands(M, N, K, b_rows, 61)
    for ea, eb in ((60, 30), (-100, 90), (-55, -50), (-70, -75), (-100, -60), (110, -120)):
        note("fp8 far scales tile %d b_rows %d fast %d 2^%d 2^%d" % (tile, b_rows, fast, ea, eb))
        x, y = (sa.double() * 2.0 ** ea).float(), (sb.double() * 2.0 ** eb).float()
        fa, fb = wide(a, x, 1), wide(b, y, b_rows)
        ref, size = fa @ fb.t(), fa.abs() @ fb.abs().t()
        low = x.double().min() * y.double().min() < 2.0 ** -126
        bound = ((128 + blocks(K) + 16) * U + (2.0 ** -11 if fast else 0)) * size
        bound = bound + (blocks(K) * 2.0 ** -125 if low else 0) + 2.0 ** -149
        bad = (product(a, x, b, y, b_rows, tile, fast) - ref).abs() - bound
        assert bad.max() <= 0, (ea, eb, float(bad.max()))


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("tile", range(-1, 11))
def test_zero_rows_and_rows_beside_an_overflow(tile, b_rows, fast):
    """Zero rows give 0 with any scale of B; a row whose product of scales overflows keeps to itself."""
    a, sa, b, sb = operands(M, N, K, b_rows, 62)
    want = product(a, sa, b, sb, b_rows, tile, fast)
    a, sa = a.clone(), sa.clone()
    a.view(torch.uint8)[::9] = 0
    sa[:, ::9] = 2.0 ** -126
    sa[2, 5] = 3e38
    sb = sb.clone()
    sb[2] *= 2.0 ** 10        # (of one block: the others as they were)
    a.view(torch.uint8)[:, 256:384][torch.arange(M) != 5] = 0
    got = product(a, sa, b, sb, b_rows, tile, fast)
    assert (got[::9] == 0).all()
    assert not got[5].isfinite().all()
    rest = torch.arange(M)[(torch.arange(M) % 9 != 0) & (torch.arange(M) != 5)]
    fa, fb = wide(a, sa, 1)[rest], wide(b, sb, b_rows)
    size = fa.abs() @ fb.abs().t()
    bound = ((128 + blocks(K) + 16) * U + (2.0 ** -11 if fast else 0)) * size
    assert ((got[rest] - fa @ fb.t()).abs() <= bound).all()
    assert want.isfinite().all()
