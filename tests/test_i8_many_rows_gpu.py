"""GPU tests of the int8 product with up to 2^31 - 1 rows, plain and grouped: a row's number plus a tile's
height passes 2^31 there.  One column and one k, so that the arrays stay at a few GB; values and
products are whole numbers of binary16, so results are held to equality."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1
GUARD = 4096
FACTORS = (3, -5, 1, 7)   # the groups' matrices


@pytest.fixture(scope="module")
def arrays():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(-128, 128, (MOST,), generator=g, dtype=torch.int8, device="cuda")
    yield dict(a=a, sa=torch.ones(MOST, device="cuda"), sb=torch.ones(4, device="cuda"),
               b=torch.tensor(FACTORS, dtype=torch.int8, device="cuda"),
               c=torch.empty(MOST + 2 * GUARD, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    lib.gemm_debug_force_i8_tile(-1)
    lib.gemm_destroy()
    torch.cuda.empty_cache()


def check(arrays, offsets, values):
    """Rows of group g are values times FACTORS[g]; everything else is as it was."""
    c = arrays["c"]
    edges = [-GUARD] + offsets + [MOST + GUARD]
    for i, (lo, hi) in enumerate(zip(edges[:-1], edges[1:])):
        for at in range(lo, hi, 1 << 28):
            end = min(hi, at + (1 << 28))
            got = c[GUARD + at:GUARD + end]
            if 0 < i < len(edges) - 2:
                assert torch.equal(got, values(at, end).half() * FACTORS[i - 1]), (i, at)
            else:
                assert (got == 77.0).all(), (i, at)


MANY = [([0, 100, MOST], tile) for tile in (-1, 0, 7, 8, 9, 10, 11)]
MANY += [(offsets, tile) for offsets in (None, [0, MOST], [5, 5, MOST - 31, MOST],
                                         [3, 2 ** 30 + 1, MOST - 1, MOST - 1, MOST]) for tile in (-1, 7, 11)]


@pytest.mark.parametrize("offsets,tile", MANY, ids=str)
def test_many_rows(arrays, offsets, tile):
    a, c = arrays["a"], arrays["c"]
    c.fill_(77.0)
    note("i8 product of 2^31 - 1 rows, offsets %s, tile %d" % (offsets, tile))
    lib.gemm_debug_force_i8_tile(tile)
    if offsets is None:
        lib.i8_gemm_bias_act(MOST, 1, 1, 1.0, a, 1, arrays["sa"], arrays["b"], 1, arrays["sb"], None, 0,
                             False, lib.TYPE_F16, c[GUARD:], 1)
    else:
        lib.i8_gemm_grouped(len(offsets) - 1, torch.tensor(offsets, dtype=torch.int32, device="cuda"), MOST,
                            1, 1, 1.0, a, 1, arrays["sa"], MOST, None, 1, arrays["b"], 1, arrays["sb"], None,
                            0, False, lib.TYPE_F16, c[GUARD:], 1)
    torch.cuda.synchronize()
    lib.gemm_debug_force_i8_tile(-1)
    check(arrays, offsets or [0, MOST], lambda lo, hi: a[lo:hi])


@pytest.mark.parametrize("tile", [-1, 7, 11])
def test_many_rows_by_index(arrays, tile):
    c, offsets = arrays["c"], [0, 100, MOST]
    index = torch.arange(MOST, dtype=torch.int32, device="cuda").remainder_(15)
    c.fill_(77.0)
    note("i8 product of 2^31 - 1 rows by index, tile %d" % tile)
    lib.gemm_debug_force_i8_tile(tile)
    lib.i8_gemm_grouped(2, torch.tensor(offsets, dtype=torch.int32, device="cuda"), MOST, 1, 1, 1.0,
                        arrays["a"], 1, arrays["sa"], 5, index, 3, arrays["b"], 1, arrays["sb"], None, 0,
                        False, lib.TYPE_F16, c[GUARD:], 1)
    torch.cuda.synchronize()
    lib.gemm_debug_force_i8_tile(-1)
    check(arrays, offsets, lambda lo, hi: arrays["a"][(index[lo:hi] // 3).long()])
