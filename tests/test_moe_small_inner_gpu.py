"""GPU tests of the binary16 mixture-of-experts layer with small inner values: whatever the size of h,
the output is held to the layer's own roundings (test_moe_gpu.py), with h itself off by half a step
of a half step of binary16, or by 2^-39 of the largest |h| of its token and expert where that is below
2^-8, else by 2^-25."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.test_fp8_gpu import activation, blocks
from tests.test_moe_gpu import U, Layer, library  # noqa: F401  (the library's lifetime)

pytestmark = pytest.mark.gpu


class Small(Layer):
    """x of token t times 2^x[t], W1 and W2 times 2^w1 and 2^w2 (by the scales, in e4m3)."""

    in_range = True      # whether the case means its output to be normal binary16 numbers

    def __init__(self, *a, xs=(), w1=0, w2=0, **kw):
        super().__init__(*a, **kw)
        for t in range(self.T):
            self.x[t] = (self.x[t].float() * 2.0 ** xs[t % len(xs)]).to(self.dtype)
        for which, by in (("1", w1), ("2", w2)):
            ws = getattr(self, "w" + which)
            if self.s1 is not None:
                getattr(self, "s" + which).mul_(2.0 ** by)
                setattr(self, "w" + which, [w * 2.0 ** by for w in ws])
            else:
                rounded = [(w * 2.0 ** by).to(self.dtype) for w in ws]
                assert all(w.isfinite().all() for w in rounded)
                setattr(self, "d" + which, self.padded(torch.stack(rounded), float("nan")))
                setattr(self, "w" + which, [w.double() for w in rounded])

    def check(self):
        T, D, I, k = self.T, self.D, self.I, self.k
        ids, p = self.ids.cpu().long(), self.w.cpu().double()
        fin = torch.finfo(self.dtype)
        half = fin.eps / 2
        for t in range(T):
            x = self.x[t].double()
            y, err, size = [torch.zeros(D, dtype=torch.float64) for _ in range(3)]
            for s in range(k):
                w1, w2 = self.w1[int(ids[t, s])], self.w2[int(ids[t, s])]
                u = w1 @ x
                du = (D + blocks(D) + 24) * U * (w1.abs() @ x.abs())
                h = activation(u[:I], self.act)
                dh = du[:I] if self.act == 0 else 1.13 * du[:I] + 2.0 ** -21 * u[:I].abs()
                if self.gated:
                    dh = u[I:].abs() * dh + h.abs() * du[I:] + dh * du[I:]
                    h = h * u[I:]
                peak = float(h.abs().max())
                floor = 2.0 ** -39 * peak if peak < 2.0 ** -8 else 2.0 ** -25
                dh = dh + 3 * U * h.abs() + half * half * h.abs() + 1.01 * floor
                y += p[t, s] * (w2 @ h)
                sz = p[t, s] * (w2.abs() @ h.abs())
                size += sz
                err += p[t, s] * (w2.abs() @ dh) + ((2 * I + blocks(I) + 24) * U + 2 * U) * sz
            err += k * U * size
            err += (y.abs() + err) * half + fin.smallest_normal * fin.eps
            got = self.y[t].cpu().double()
            assert (got[D:] == 77.0).all(), "written past the end"
            bad = (got[:D] - y).abs() - err
            assert got[:D].isfinite().all() and bad.max() <= 0, (t, int(bad.argmax()), float(bad.max()))
            assert not self.in_range or y.abs().median() > 2.0 ** -14


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [1, 3, 20, 40])
def test_small_rows(T, gated, fp8):
    """h of about 2^-20; lengths with and without a ragged end."""
    for D, I in ((200, 83), (128, 256), (64, 7), (40, 1100)):
        by = -9 if gated else -18
        Small(T, D, I, 5, 2, "f16", fp8, gated=gated, act=lib.ACT_SILU if gated else lib.ACT_NONE,
              seed=51, xs=(by if gated else 0,), w1=0 if gated else by + 8 * (not fp8),
              w2=24 if fp8 else 14, size=0.3 if D < 100 else 0.05).run()


@pytest.mark.parametrize("rows", [16, 32, 64])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [5, 20, 40])
def test_small_and_ordinary_rows_share_experts(T, fp8, rows):
    """Every third token small, in tiles of every width; the others as without it, bit for bit."""
    assert lib.gemm_debug_force_moe_rows(rows) == lib.STATUS_SUCCESS
    try:
        m = Small(T, 201, 300, 3, 2, "f16", fp8, seed=52, xs=(0, -10, 0), w2=4, norm=False)
        m.buffers()
        m.call()
        torch.cuda.synchronize()
        mixed = m.y.clone()
        small = torch.arange(T) % 3 == 1
        for t in range(T):
            if small[t]:
                m.dx[t, :201] = m.dx[t, :201].float().mul(2.0 ** 10).to(m.dtype)
        m.call()
        torch.cuda.synchronize()
        assert torch.equal(m.y[~small], mixed[~small])
        m.in_range = False
        m.run()
    finally:
        lib.gemm_debug_force_moe_rows(0)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("by", [-60, -100])
def test_scales_far_apart(T, by):
    """e4m3 weights whose scales bring h far below binary16 and the output back."""
    Small(T, 130, 150, 3, 2, "f16", True, gated=False, act=lib.ACT_NONE, seed=53, xs=(0,), w1=by,
          w2=-by).run()


def test_zero_rows():
    m = Small(4, 96, 64, 6, 2, "f16", seed=54, xs=(0, -10))
    m.x[2] = 0
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    assert (m.y[2, :96] == 0).all() and m.y[:, :96].isfinite().all()


@pytest.mark.parametrize("T", [3, 33])
def test_infinite_weight_of_a_small_row(T):
    m = Small(T, 77, 45, 1, 1, "f16", gated=False, act=lib.ACT_NONE, seed=55, xs=(-20,))
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    clean = m.y[:, :77].clone()
    m.d2[0, 9, 40] = float("inf")
    m.call()
    torch.cuda.synchronize()
    h = m.x.double() @ m.w1[0][40]
    sure = h.abs() > 80 * U * (m.x.double().abs() @ m.w1[0][40].abs())
    got = m.y[:, :77].cpu()
    assert torch.equal(got[sure, 9].double(), h.sign()[sure] * float("inf"))
    got[:, 9] = clean[:, 9].cpu()
    assert torch.equal(got, clean.cpu())


def test_small_rows_in_a_graph():
    m = Small(4, 128, 200, 4, 2, "f16", seed=56, xs=(-10, 0), w2=10)
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.call()
    for by in (0.0, -10.0, 3.0):
        m.dx[:, :128] = (m.x.float() * 2.0 ** by).to(m.dtype).cuda()
        m.call()
        torch.cuda.synchronize()
        want = m.y.clone()
        m.y.zero_()
        m.ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.y, want)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 3), (3, 1, 1), (40, 4, 2)])
def test_infinite_weight_of_a_value_that_rounds_to_zero(T, E, k):
    """h of one column is below 2^-25 in a row of ordinary size: its product with an infinite weight is
    infinite all the same."""
    m = Layer(T, 77, 45, E, k, "f16", gated=False, act=lib.ACT_NONE, seed=57, size=1.0)
    m.x = (m.x.abs().float() * 2.0 ** -8).half()
    m.w1 = [w.clone() for w in m.w1]
    for w in m.w1:
        w[40] = -(2.0 ** -24)
    m.d1[:, 40, :77] = -(2.0 ** -24)
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    clean = m.y[:, :77].clone()
    assert clean.isfinite().all()
    m.d2[:, 9, 40] = float("-inf")
    m.call()
    torch.cuda.synchronize()
    got = m.y[:, :77]
    assert (got[:, 9] == float("inf")).all()
    got[:, 9] = clean[:, 9]
    assert torch.equal(got, clean)
