"""GPU tests of the int8 product's alpha far from one: it counts as a factor like the scales, so that no
order of the four factors under- or overflows before their product does.

Bounds are those of tests/test_i8_gpu.py: alpha's multiplication is the fourth of its four roundings, with
the bias in the same one."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_i8_gpu import Product, padded, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_debug_force_i8_tile(-1)
    lib.gemm_destroy()


def far(alpha, ea, eb, **options):
    p = Product(9, 40, 200, pad=1, alpha=alpha, **options)
    p.sa, p.sb = torch.full((9,), 2.0 ** ea * 1.25), torch.full(p.sb.shape, 2.0 ** eb * 1.5)
    p.dsa, p.dsb = p.sa.cuda(), p.sb.cuda()
    return p


# (log2 of alpha, of the rows' and of the channels' scales; the sums are up to 2^21)
FAR = [(100, -80, -80), (60, -100, -60), (-60, 70, 70), (-100, 90, 90), (127, -126, -120), (-126, 120, 100),
       (-147, 127, 127), (40, -70, -75), (40, -120, -20), (20, -126, -20), (60, 40, 20), (126, -140, -90)]


@pytest.mark.parametrize("tile", range(-1, 12))
@pytest.mark.parametrize("e,ea,eb", FAR)
def test_far_alpha(e, ea, eb, tile):
    for alpha in (2.0 ** e, -1.375 * 2.0 ** e if e > -120 else -(2.0 ** e)):
        for rows in (None, [4, 0, 5]):
            note("i8 product alpha %g scales 2^%d 2^%d tile %d rows %s" % (alpha, ea, eb, tile, rows))
            run(far(alpha, ea, eb, type_="f32", bias=False, rows=rows), tile)


@pytest.mark.parametrize("tile", range(-1, 12))
def test_far_alpha_with_bias_activation_and_gate(tile):
    for options in (dict(type_="f32"), dict(type_="bf16", act=1), dict(type_="f32", act=2, gated=True),
                    dict(type_="f16", gated=True)):
        for e, ea, eb in ((100, -70, -45), (-100, 60, 25), (60, -100, 25)):   # values about one
            note("i8 product alpha 2^%d tile %d %s" % (e, tile, options))
            run(far(1.375 * 2.0 ** e, ea, eb, **options), tile)


@pytest.mark.parametrize("tile", range(-1, 12))
def test_alpha_that_is_not_finite(tile):
    """An infinite alpha: infinities of the sums' signs, and NaN where a sum is zero."""
    p = Product(9, 40, 200, pad=1, type_="f32", alpha=float("inf"))
    p.a[4] = 0
    p.da = padded(p.a, p.ld)
    sums = p.a.double() @ p.b[0].double().t()
    for alpha in (float("inf"), float("-inf"), float("nan")):
        p.alpha = alpha
        lib.gemm_debug_force_i8_tile(tile)
        note("i8 product alpha %g tile %d" % (alpha, tile))
        p.call()
        torch.cuda.synchronize()
        lib.gemm_debug_force_i8_tile(-1)
        assert torch.equal(torch.nan_to_num(p.c.cpu()[:9, :40].double(), 5.0),
                           torch.nan_to_num(alpha * sums, 5.0))
