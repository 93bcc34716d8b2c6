"""GPU test of block quantisation of 16-bit values at the ties: held to the definition (scale and
quotient in fp32), and to the quotient in exact arithmetic wherever that is no tie."""
import pytest
import torch

from tests.gpu_helpers import note
from tests.test_fp8_gpu import E4M3, TYPES, library, reference, run_quantize  # noqa: F401

pytestmark = pytest.mark.gpu


def pairs(type_):
    """Rows of one block: the largest value m, and 127 values of equal or smaller exponent; every pair of
    bfloat16 significands at 17 exponents, and as many of binary16."""
    n = torch.arange(128) if type_ == "bf16" else torch.arange(128) * 8 + 5
    f = 1 + n.double() / (128 if type_ == "bf16" else 1024)
    rows = []
    for e in range(17):
        x = torch.cat([f[:, None], (f * 2.0 ** -e).expand(128, 128)[:, :127]], 1)
        if e == 0:
            x = torch.minimum(x, x[:, :1])      # (nothing above the row's own largest)
        rows.append(x)
    x = torch.cat(rows) * 32.0
    assert torch.equal(x.to(TYPES[type_][0]).double(), x)
    return x.to(TYPES[type_][0])


def quotients(x):
    y = x.double().reshape(x.shape[0], -1, 128)
    return (y * 448 / y.abs().amax(2, keepdim=True)).reshape(x.shape)


def ideal(x):
    q = quotients(x)
    space = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / space) * space).float().to(E4M3)


@pytest.mark.parametrize("type_", ["bf16", "f16"])
def test_pairs_of_significands(type_):
    note("quantize pairs %s" % type_)
    x = pairs(type_)
    got, turned = run_quantize(x, 1)
    q, s = reference(x, 1)
    assert torch.equal(got[1], s) and torch.equal(got[0].view(E4M3).float(), q.float())
    assert torch.equal(turned[0].view(E4M3).float(), reference(x.t(), 1)[0].float())
    # Off the ties (by less than the two roundings of fp32) it is the exact quotient's rounding.
    e = quotients(x)
    r = e / torch.exp2(torch.floor(torch.log2(e.abs().clamp(min=2.0 ** -6))) - 3)
    tie = ((r - torch.floor(r)) - 0.5).abs() <= 2.0 ** -23 * r
    assert torch.equal(got[0].view(E4M3).float()[~tie], ideal(x).float()[~tie])


def test_the_tie_of_the_header():
    x = torch.zeros((1, 128), dtype=torch.bfloat16)
    x[0, :2] = torch.tensor([62.0, 2.90625])
    got, _ = run_quantize(x, 1, turned=False)
    assert got[0].view(E4M3).float()[0, :2].tolist() == [448.0, 22.0]


@pytest.mark.parametrize("b", [1, 128])
@pytest.mark.parametrize("type_", ["bf16", "f16"])
def test_fp32_ties_go_to_even(type_, b):
    """fp32 inputs are divided by the scale before it is rounded: the same pairs, held in fp32, are the
    exact quotient's rounding everywhere."""
    note("quantize fp32 pairs %s block %d" % (type_, b))
    x = pairs(type_).float()
    if b == 128:     # one row a block
        x = torch.nn.functional.pad(x[::7, None], (0, 0, 0, 127)).reshape(-1, 128)
    kept = slice(None) if b == 1 else slice(None, None, 128)
    (got, s), turned = run_quantize(x, b)
    assert torch.equal(s, reference(x, b)[1])
    want = ideal(x[kept]).float()
    assert torch.equal(got[kept].view(E4M3).float(), want)
    if b == 128:     # (along columns the blocks of 1 x 128 are others)
        assert torch.equal(turned[0].t()[kept].contiguous().view(E4M3).float(), want)
    else:
        (_, other) = run_quantize(x.t().contiguous(), 1)
        assert torch.equal(other[0].view(E4M3).float(), want)
