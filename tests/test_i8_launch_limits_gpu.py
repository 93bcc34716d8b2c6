"""GPU tests of calls with more work than a launch has workgroups for, where the kernels loop: rows to
quantise, tokens to exchange, and a product with more output tiles than the tiled kernels take.  Values are
small whole numbers and powers of two, so that every result is exact and held to equality."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_destroy()
    torch.cuda.empty_cache()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("rows,cols", [(2 ** 22 + 5, 24), (2 ** 20 + 3, 4104)])
def test_rows_to_quantise(rows, cols):
    g = generator(rows)
    q = torch.randint(-127, 128, (rows, cols), generator=g, dtype=torch.int8, device="cuda")
    q[:, cols // 2] = 127
    s = torch.exp2(torch.randint(-3, 4, (rows,), generator=g, device="cuda").float())
    x = q.to(torch.bfloat16).mul_(s.bfloat16()[:, None])
    got = torch.full((rows + 1, cols), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), -7.0, device="cuda")
    note("i8_quantize %dx%d" % (rows, cols))
    lib.i8_quantize(rows, cols, lib.TYPE_BF16, x, cols, got, cols, scale)
    torch.cuda.synchronize()
    assert torch.equal(scale[:rows], s) and float(scale[rows]) == -7.0
    assert torch.equal(got[:rows], q) and (got[rows] == 77).all()


def test_tokens_to_exchange():
    T, k, cols = 2 ** 22 + 9, 2, 8
    g = generator(3)
    pos = torch.randperm(T * k, generator=g, device="cuda").int().view(T, k)
    at = pos.long()
    w = torch.exp2(torch.randint(-2, 3, (T, k), generator=g, device="cuda").float())
    x = torch.randint(-8, 9, (T, cols), generator=g, device="cuda").float()
    y = torch.full((T * k + 1, cols), 77.0, device="cuda")
    note("exchange of %d tokens" % T)
    lib.moe_dispatch(T, k, cols, lib.TYPE_F32, x, cols, pos, w, y, cols, T * k)
    torch.cuda.synchronize()
    assert torch.equal(y[at], w[..., None] * x[:, None]) and (y[T * k] == 77.0).all()
    rows = torch.randint(-8, 9, (T * k, cols), generator=g, device="cuda").float()
    z = torch.full((T + 1, cols), 77.0, device="cuda")
    lib.moe_combine(T, k, cols, lib.TYPE_F32, rows, cols, T * k, pos, w, z, cols)
    torch.cuda.synchronize()
    assert torch.equal(z[:T], (w[..., None] * rows[at]).sum(1)) and (z[T] == 77.0).all()
    dw = torch.full((T * k + 1,), 77.0, device="cuda")
    y.fill_(77.0)
    lib.moe_combine_grad(T, k, cols, lib.TYPE_F32, x, cols, rows, cols, T * k, pos, w, y, cols, dw)
    torch.cuda.synchronize()
    assert torch.equal(y[at], w[..., None] * x[:, None]) and (y[T * k] == 77.0).all()
    assert torch.equal(dw[:-1].view(T, k), (x[:, None] * rows[at]).sum(2)) and float(dw[-1]) == 77.0


def test_tiles_of_a_product():
    """More than 2^23 tiles of 32 x 64: 34 GB of results."""
    M, N, K = 2 ** 17 + 40, 2 ** 17 + 72, 16
    g = generator(4)
    a = torch.randint(-11, 12, (M, K), generator=g, dtype=torch.int8, device="cuda")
    b = torch.randint(-11, 12, (N, K), generator=g, dtype=torch.int8, device="cuda")
    c = torch.full((M + 1, N), 77.0, dtype=torch.float16, device="cuda")
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    note("i8 product %dx%dx%d" % (M, N, K))
    lib.i8_gemm_bias_act(M, N, K, 1.0, a, K, sa, b, K, sb, None, 0, False, lib.TYPE_F16, c, N)
    torch.cuda.synchronize()
    assert (c[M] == 77.0).all()
    bt = b.float().t().contiguous()
    for at in range(0, M, 4096):
        end = min(M, at + 4096)
        assert torch.equal(c[at:end].float(), a[at:end].float() @ bt), at
