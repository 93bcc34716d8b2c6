"""GPU tests of every kernel instance of the mixture-of-experts layer against its definition in 64
bits (the bound and the layer: test_moe_gpu.py): all tile widths at each number of tokens, rows long
enough that every wave takes several blocks of columns, and the ways to find an expert's tokens with few
and with many experts."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.test_moe_gpu import Layer, library  # noqa: F401  (the library's lifetime)

pytestmark = pytest.mark.gpu


@pytest.fixture
def rows(request):
    assert lib.gemm_debug_force_moe_rows(request.param) == lib.STATUS_SUCCESS
    yield request.param
    lib.gemm_debug_force_moe_rows(0)


@pytest.mark.parametrize("rows", [16, 32, 64], indirect=True)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [5, 20, 40])
def test_every_tile_width(T, gated, fp8, rows):
    """Ragged rows and columns; the second half of W1 starts inside a block of 128 rows, a fragment
    of 16 rows lies in two."""
    Layer(T, 201, 83, 5, 2, "bf16", fp8, gated=gated, pad=3, seed=31).run()
    Layer(T, 333, 300, 3, 3, "f16", fp8, act=lib.ACT_GELU_TANH, gated=gated, norm=False,
          seed=32).run()
    Layer(T, 256, 256, 2, 1, "bf16", fp8, act=lib.ACT_NONE, gated=gated, seed=33).run()


@pytest.mark.parametrize("rows", [0, 16, 64], indirect=True)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,I", [(4300, 40), (40, 4300), (2048, 64), (64, 2048)])
@pytest.mark.parametrize("T", [1, 3, 20, 40])
def test_several_blocks_of_columns_per_wave(T, D, I, fp8, rows):
    Layer(T, D, I, 6, 4, "bf16", fp8, seed=34, size=0.02).run()
    Layer(T, D, I, 3, 2, "f16", fp8, act=lib.ACT_GELU_TANH, gated=False, seed=35, size=0.02).run()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (1, 130, 32), (20, 129, 6), (40, 200, 4),
                                   (40, 256, 6), (64, 256, 3)])
def test_grid_of_pairs(T, E, k, fp8):
    assert T * k < E <= 256
    Layer(T, 70, 36, E, k, "bf16", fp8, seed=36).run()
    Layer(T, 70, 36, E, k, "f16", fp8, gated=False, norm=False, seed=37).run()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 257, 8), (1, 384, 8), (1, 1024, 32), (4, 384, 8),
                                   (20, 1024, 8), (64, 257, 2), (64, 1024, 32)])
def test_many_experts(T, E, k, fp8):
    Layer(T, 70, 36, E, k, "bf16", fp8, seed=38).run()
    Layer(T, 70, 36, E, k, "f16", fp8, gated=False, norm=False, seed=39).run()


def test_equal_logits_of_many_experts():
    for T, E, k in ((1, 256, 8), (2, 700, 9)):
        m = Layer(T, 64, 32, E, k, seed=40)
        m.r[:] = m.r[0].clone()
        m.r[E // 2:] *= 2
        m.run()
        want = torch.where(m.x.double() @ m.r[0].double() > 0, E // 2, 0)
        assert torch.equal(m.ids.cpu().long(), want[:, None] + torch.arange(k))
