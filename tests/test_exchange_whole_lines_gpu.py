"""GPU tests of the exchange's rows of whole 128-byte lines, which combine and its gradient load past the
caches, and of the same widths with a base or a distance of rows that breaks the lines; up to several
workgroups a row and more slots than are loaded together.  Bounds are those of test_exchange_gpu.py."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_exchange_gpu import Exchange
from tests.test_i8_gpu import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_destroy()


def shifted(x):
    """The same values a step of the type behind a 128-byte line."""
    out = torch.empty(x.numel() + 64, dtype=x.dtype, device="cuda")
    assert out.data_ptr() % 128 == 0
    out = out[1:1 + x.numel()].view(x.shape)
    out.copy_(x)
    return out


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("lines", ["whole", "distance", "base"])
@pytest.mark.parametrize("T,k,cols", [(1, 1, 64), (9, 3, 64), (33, 8, 512), (12, 9, 512), (300, 8, 4096),
                                      (7, 17, 4096), (5, 6, 8192), (3, 32, 16384)])
def test_widths_of_whole_lines(T, k, cols, lines, type_):
    for weighted in (True, False):
        e = Exchange(T, k, cols, type_, weighted=weighted, pad=1 if lines == "distance" else 0,
                     seed=T + k + cols)
        if lines == "base":
            e.dsorted, e.dtokens = shifted(e.dsorted), shifted(e.dtokens)
        else:
            assert e.dsorted.data_ptr() % 128 == 0
        note("exchange %dx%d cols %d %s weighted %s, %s" % (T, k, cols, type_, weighted, lines))
        e.dispatch()
        e.combine()
        torch.cuda.synchronize()
        e.check_dispatch()
        e.check_combine()
        for dx, dw in ((True, True), (True, False), (False, True)):
            e.grad(dx, dw)
            torch.cuda.synchronize()
            e.check_grad()


@pytest.mark.parametrize("type_", list(TYPES))
def test_lines_do_not_change_results(type_):
    """The two ways of loading give the same bits."""
    e = Exchange(40, 9, 1024, type_, seed=3)
    e.combine()
    e.grad()
    z, gx, gw = e.z, e.gx, e.gw
    e.dsorted = shifted(e.dsorted)
    note("exchange of 1024 columns %s, both ways" % type_)
    e.combine()
    e.grad()
    torch.cuda.synchronize()
    assert torch.equal(z, e.z) and torch.equal(gx, e.gx) and torch.equal(gw, e.gw)
