"""GPU test of block quantisation of bfloat16 blocks of tiny values, whose remainders x - q s lie
below fp32's smallest number: held to the definition like any other (binary16 cannot hold such blocks, and
fp32 inputs are divided in 64 bits)."""
import pytest
import torch

from tests.gpu_helpers import note
from tests.test_fp8_gpu import E4M3, library, reference, run_quantize  # noqa: F401

pytestmark = pytest.mark.gpu


def test_tiny_blocks():
    """Every bfloat16 number m from 2^-133 to 2^-90 as the largest of a row of numbers down to 2^-19 m."""
    bits = torch.arange(1, 0x7F80, dtype=torch.int32)
    v = (bits << 16).view(torch.float32).double()
    m = v[v < 2.0 ** -90]
    x = m[:, None] * (0.5 + torch.rand((len(m), 128), generator=torch.Generator().manual_seed(1)).double())
    x = x * torch.exp2(-torch.randint(0, 20, x.shape, generator=torch.Generator().manual_seed(2)).double())
    x = torch.minimum(x, m[:, None])
    x[:, 0] = m
    # The pairs that went to the wrong neighbour.
    for i, (big, small) in enumerate([(5.830451980078546e-36, 8.540701142693183e-39),
                                      (6.488728816539027e-36, 3.801989540940836e-38),
                                      (7.147005652999508e-36, 5.234623281005499e-39)]):
        x[i] = small
        x[i, 0] = big
    x = x.float().to(torch.bfloat16)
    note("quantize tiny blocks %d" % len(m))
    got, turned = run_quantize(x, 1)
    q, s = reference(x, 1)
    assert torch.equal(got[1], s)
    assert torch.equal(got[0].view(E4M3).float(), q.float())
    y = x.t().contiguous()
    plain, other = run_quantize(y, 1)
    assert torch.equal(other[0], got[0]) and torch.equal(other[1], s)


@pytest.mark.parametrize("b", [1, 128])
def test_blocks_beside_larger_ones(b):
    """Tiny, ordinary and large blocks side by side."""
    x = torch.randn((300, 384), generator=torch.Generator().manual_seed(3)).double()
    x[:, :128] *= 2.0 ** -118
    x[128:256, 256:] *= 2.0 ** 110
    x[::7, 256:] *= 2.0 ** -64
    x = x.float().to(torch.bfloat16)
    for got, m in zip(run_quantize(x, b), (x, x.t())):
        q, s = reference(m, b)
        assert torch.equal(got[1], s) and torch.equal(got[0].view(E4M3).float(), q.float())
