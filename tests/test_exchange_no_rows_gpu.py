"""GPU tests of the exchange's calls that have no sorted rows (or no columns): pointers that such a call may
leave null are not read, and what is documented as zero is zero."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
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


def entries(T, k, kind):
    n = {"lost": torch.full((T, k), -1), "past": torch.arange(T * k).view(T, k)}[kind]
    return n.int().cuda()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("kind", ["lost", "past"])   # entries of no expert; rows that are all past the end
@pytest.mark.parametrize("T,k,cols,x_rows", [(1, 1, 1, 0), (5, 3, 100, 0), (40, 8, 4096, 0), (7, 9, 20001, 0),
                                             (3, 32, 512, 0), (6, 4, 0, 0), (6, 4, 0, 24)])
def test_gradients_without_rows(T, k, cols, x_rows, kind, type_):
    dtype, code = TYPES[type_]
    pos = entries(T, k, kind)
    w = torch.full((T, k), float("nan"), device="cuda")   # (not read for entries that are skipped)
    for weights in (w, None):
        for out in (torch.full((3, max(cols, 1)), 77.0, dtype=dtype, device="cuda"), None):
            dw = torch.full((T * k + 1,), 77.0, device="cuda")
            note("combine_grad %dx%d cols %d x_rows %d %s, null dY" % (T, k, cols, x_rows, type_))
            lib.moe_combine_grad(T, k, cols, code, None, cols + 1, None, cols + 1, x_rows, pos, weights, out,
                                 cols + 1, dw)
            torch.cuda.synchronize()
            assert not dw[:-1].any() and float(dw[-1]) == 77.0
            assert out is None or (out == 77.0).all()
    out = torch.full((3, max(cols, 1)), 77.0, dtype=dtype, device="cuda")
    lib.moe_combine_grad(T, k, cols, code, None, cols + 1, None, 0, x_rows, pos, w, out, cols + 1, None)
    torch.cuda.synchronize()
    assert (out == 77.0).all()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("T,k,cols", [(1, 1, 3), (5, 9, 100), (40, 8, 4096)])
def test_combine_and_dispatch_without_rows(T, k, cols, type_):
    dtype, code = TYPES[type_]
    pos = entries(T, k, "past")
    y = torch.full((T + 1, cols), 77.0, dtype=dtype, device="cuda")
    note("combine, dispatch %dx%d cols %d %s without rows" % (T, k, cols, type_))
    lib.moe_combine(T, k, cols, code, None, cols, 0, pos, None, y, cols)
    lib.moe_dispatch(T, k, cols, code, None, cols, pos, None, None, cols, 0)
    torch.cuda.synchronize()
    assert not y[:T].any() and (y[T] == 77.0).all()


def test_gradients_without_rows_in_a_graph():
    T, k = 20, 6
    pos, dw = entries(T, k, "past"), torch.full((T * k,), 77.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    note("combine_grad without rows, captured")
    with torch.cuda.graph(graph):
        lib.moe_combine_grad(T, k, 300, lib.TYPE_BF16, None, 300, None, 300, 0, pos, None, None, 0, dw)
    for _ in range(3):
        dw.fill_(77.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not dw.any()
