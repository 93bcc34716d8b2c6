"""GPU tests of row numbers outside A in the grouped int8 product: a number past the end is the last row
of A, a negative one row 0, as documented; padding's -1 of a sort among them."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_i8_gpu import Product, run

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


@pytest.mark.parametrize("tile", range(-1, 12))
@pytest.mark.parametrize("gather,per", [(7, 2), (7, 1), (1, 1), (1, 5), (300, 2 ** 31 - 1)])
def test_rows_outside_a(gather, per, tile):
    for pad, off, K in ((1, 0, 100), (1, 0, 300), (0, 3, 130)):
        p = Product(150, 50, K, rows=[60, 0, 1, 89], gather=gather, pad=pad, off=off, act=2,
                    type_="f32", gated=True)
        p.per = per
        most = gather * per
        numbers = [-1, -7, -2 ** 31, 0, per - 1, most - 1, most, most + 1, 2 ** 31 - 1]
        given = torch.tensor([min(n, 2 ** 31 - 1) for n in numbers], dtype=torch.int64)[torch.arange(150) % 9]
        p.dindex = given.int().cuda()
        # (What check reads: the row meant, times per.)
        p.index = torch.div(given.clamp_min(0), per, rounding_mode="floor").clamp_max(gather - 1) * per
        note("i8 grouped, rows outside A: %d rows, per %d, tile %d, K %d" % (gather, per, tile, K))
        run(p, tile)
