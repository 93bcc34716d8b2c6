"""A layer of experts over a prompt, as the int8 operators make it: tokens quantised, sorted by expert, the
gated up projection reading them where they lie, its results quantised, the down projection, and
back to the tokens with the router's weights.  Every step is held to its own definition on what the step
before it left, with the tolerances of the steps' own tests; and the whole to the layer in 64 bits."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_exchange_gpu import reference_sort
from tests.test_i8_gpu import U, activation, reference_product, reference_rows

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_destroy()


class Experts:
    def __init__(self, T, D, I, E, k, lost=0.1, seed=0):
        self.__dict__.update(T=T, D=D, I=I, E=E, k=k)
        g = torch.Generator().manual_seed(seed)
        self.w1 = torch.randn((E * 2 * I, D), generator=g) * D ** -0.5
        self.w2 = torch.randn((E * D, I), generator=g) * I ** -0.5
        self.buffers()
        for name, w, cols in (("1", self.w1, D), ("2", self.w2, I)):
            q = torch.empty((len(w), cols), dtype=torch.int8, device="cuda")
            s = torch.empty(len(w), device="cuda")
            lib.i8_quantize(len(w), cols, lib.TYPE_F32, w.cuda(), cols, q, cols, s)
            setattr(self, "q" + name, q)
            setattr(self, "s" + name, s)
        self.inputs(seed, lost)

    def inputs(self, seed, lost):
        g = torch.Generator().manual_seed(100 + seed)
        x = torch.randn((self.T, self.D), generator=g).to(BF16)
        p, ids = torch.softmax(torch.randn((self.T, self.E), generator=g), 1).topk(self.k)
        out = torch.rand((self.T, 1), generator=g) < lost
        self.x_host, self.ids_host = x, ids.masked_fill(out, -1).int()
        self.w_host = p / p.sum(1, keepdim=True)
        self.x.copy_(x)
        self.ids.copy_(self.ids_host)
        self.w.copy_(self.w_host)

    def buffers(self):
        T, D, I, E, R = self.T, self.D, self.I, self.E, self.T * self.k

        def empty(*shape, dtype=torch.float32):
            return torch.zeros(shape, dtype=dtype, device="cuda")
        self.x, self.ids, self.w = empty(T, D, dtype=BF16), empty(T, self.k, dtype=torch.int32), empty(T, self.k)
        self.qx, self.sx = empty(T, D, dtype=torch.int8), empty(T)
        self.offsets, self.src = empty(E + 1, dtype=torch.int32), empty(R, dtype=torch.int32)
        self.pos = empty(T, self.k, dtype=torch.int32)
        self.h, self.qh, self.sh = empty(R, I, dtype=BF16), empty(R, I, dtype=torch.int8), empty(R)
        self.y, self.out = empty(R, D, dtype=BF16), empty(T, D, dtype=BF16)
        self.ws = empty(lib.moe_sort_workspace(T, self.k, E), dtype=torch.uint8)

    def __call__(self):
        T, D, I, E, k = self.T, self.D, self.I, self.E, self.k
        R = T * k
        lib.i8_quantize(T, D, lib.TYPE_BF16, self.x, D, self.qx, D, self.sx)
        lib.moe_sort(T, k, E, self.ids, self.offsets, self.src, self.pos, self.ws, self.ws.numel())
        lib.i8_gemm_grouped(E, self.offsets, R, I, D, 1.0, self.qx, D, self.sx, T, self.src, k, self.q1, D,
                            self.s1, None, lib.ACT_SILU, True, lib.TYPE_BF16, self.h, I)
        lib.i8_quantize(R, I, lib.TYPE_BF16, self.h, I, self.qh, I, self.sh)
        lib.i8_gemm_grouped(E, self.offsets, R, D, I, 1.0, self.qh, I, self.sh, R, None, 1, self.q2, I,
                            self.s2, None, lib.ACT_NONE, False, lib.TYPE_BF16, self.y, D)
        lib.moe_combine(T, k, D, lib.TYPE_BF16, self.y, D, R, self.pos, self.w, self.out, D)

    def check(self):
        T, D, I, E, k = self.T, self.D, self.I, self.E, self.k
        cpu = {n: getattr(self, n).cpu() for n in ("qx", "sx", "offsets", "src", "pos", "h", "qh", "sh", "y",
                                                   "out", "q1", "s1", "q2", "s2")}
        q, s = reference_rows(self.x_host)
        assert torch.equal(cpu["qx"], q) and torch.equal(cpu["sx"], s)
        offsets, src, pos = reference_sort(self.ids_host, E)
        assert torch.equal(cpu["offsets"], offsets) and torch.equal(cpu["src"], src)
        assert torch.equal(cpu["pos"].flatten(), pos)
        n = int(offsets[-1])
        q, s = reference_rows(cpu["h"])
        assert torch.equal(cpu["qh"][:n], q[:n]) and torch.equal(cpu["sh"][:n], s[:n])
        for e in range(E):
            lo, hi = offsets[e:e + 2].tolist()
            read = src[lo:hi].long() // k
            for got, a, sa, b, sb, rows, act, gated in (
                    (cpu["h"], cpu["qx"][read], cpu["sx"][read], cpu["q1"], cpu["s1"], 2 * I, lib.ACT_SILU, True),
                    (cpu["y"], cpu["qh"][lo:hi], cpu["sh"][lo:hi], cpu["q2"], cpu["s2"], D, 0, False)):
                want, bound = reference_product(a, sa, b[e * rows:(e + 1) * rows], sb[e * rows:(e + 1) * rows],
                                                1.0, None, act, gated, BF16)
                assert ((got[lo:hi].double() - want).abs() <= bound).all()
        valid = cpu["pos"] >= 0
        w = torch.where(valid, self.w_host, 0.0).double()[..., None]
        parts = w * cpu["y"].double()[cpu["pos"].clamp_min(0).long()]
        want, size = parts.sum(1), parts.abs().sum(1)
        bound = (k + 1) * U * size + 2.0 ** -8 * (want.abs() + k * U * size) + 1e-40
        assert ((cpu["out"].double() - want).abs() <= bound).all()

    def relative_error(self):
        """Against the layer in 64 bits with the weights as they were."""
        y = torch.zeros((self.T, self.D), dtype=torch.float64)
        w1, w2 = self.w1.double().view(self.E, 2 * self.I, self.D), self.w2.double().view(self.E, self.D, self.I)
        for e in range(self.E):
            t, s = torch.nonzero(self.ids_host == e, as_tuple=True)
            u = self.x_host.double()[t] @ w1[e].t()
            h = activation(u[:, :self.I], lib.ACT_SILU) * u[:, self.I:]
            y.index_add_(0, t, (h @ w2[e].t()) * self.w_host.double()[t, s, None])
        return float((self.out.cpu().double() - y).norm() / y.norm())


@pytest.mark.parametrize("T,D,I,E,k", [(1, 256, 128, 8, 2), (5, 200, 77, 60, 6), (130, 512, 256, 8, 2),
                                       (700, 384, 136, 16, 4), (64, 64, 33, 4, 4)])
def test_layer(T, D, I, E, k):
    """The rounding to int8 of a normal row of n values is off by a uniform error of s = max / 127, as a norm
    s / sqrt(12) a value: with max <= sqrt(2 ln(2 n)) + 1 below 5 deviations, at most 5 / 127 / sqrt(12)
    = 0.0114 of the row.  The gated inner values have a longer tail: a max of at most 25 of their
    deviations over the rows here, 0.057.  Two operands for the first product (its two sums' errors reach
    h through both factors: twice 0.0114 sqrt 2), two for the second: 0.032 + 0.057 + 0.0114 = 0.1 at
    most, if the parts added up, and bfloat16's 2^-8 beside them."""
    note("int8 experts %dx%d I %d E %d k %d" % (T, D, I, E, k))
    layer = Experts(T, D, I, E, k, lost=0.1 if T > 1 else 0.0)
    layer()
    torch.cuda.synchronize()
    layer.check()
    assert layer.relative_error() <= 0.11


def test_layer_from_a_graph():
    """Captured once, replayed with other tokens and other routes, eager work between."""
    layer, other = Experts(90, 256, 128, 8, 2), Experts(33, 128, 64, 4, 2, seed=9)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for i in range(4):
        layer.inputs(i, 0.3)
        layer.out.fill_(7.0)
        other.inputs(i, 0.0)
        other()
        graph.replay()
        other()
        torch.cuda.synchronize()
        layer.check()
        other.check()


def test_two_layers_on_two_streams():
    a, b = Experts(300, 256, 128, 8, 2, seed=1), Experts(250, 384, 96, 16, 3, seed=2)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            a()
        with torch.cuda.stream(sb):
            b()
    torch.cuda.synchronize()
    a.check()
    b.check()
