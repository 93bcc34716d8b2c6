"""GPU test that block quantisation keeps the sign of a zero: x / s of -0 is -0, byte 0x80."""
import pytest
import torch

from tests.test_fp8_gpu import TYPES, library, matrix, reference, run_quantize  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type_", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b", [1, 128])
def test_negative_zero(b, type_):
    x = matrix(130, 260, type_, 41)
    x[::3, ::2] = -0.0
    x[1::3, 1::2] = 0.0
    x[50] = -0.0                      # a row, and below a whole block, of nothing else
    x[:, 128:256] = -0.0
    x[:, 256:] *= torch.tensor(1e-4)  # (some that round to a zero of their own sign)
    got = run_quantize(x, b)
    for (q, _), m in zip(got, (x, x.t())):
        assert torch.equal(q, reference(m, b)[0].view(torch.uint8))
    alone = run_quantize(x, b, turned=False)[0][0]
    assert torch.equal(alone, got[0][0])
