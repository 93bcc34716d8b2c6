"""GPU tests of the few-token mixture-of-experts layer against its definition in 64 bits.

The choice of experts is held to equality.  The output is held to a bound made of the layer's own
roundings, u = 2^-24, carried through it element by element:
  u-products   - (D + D / 128 + 24) u of sum |x||w1|;
  activation   - a slope of at most 1.13 and 2^-21 |x|;
  h            - 3 u |h| (product, clamp), then held as two 16-bit numbers: half a step of a half step
                 of the type, and in binary16 never closer than 2^-25;
  down product - (2 I + I / 128 + 24) u of sum |h||w2|, the weights' 2 u, the sum over slots;
  result       - half a step of its type."""
import math

import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_fp8_gpu import E4M3, activation, blocks, reference

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f16": (torch.float16, lib.TYPE_F16), "bf16": (torch.bfloat16, lib.TYPE_BF16)}


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_destroy()


class Layer:
    def __init__(self, T, D, I, E, k, type_="bf16", fp8=False, act=lib.ACT_SILU, gated=True,
                 norm=True, pad=0, seed=0, size=0.05, logits=1.5):
        self.__dict__.update(T=T, D=D, I=I, E=E, k=k, act=act, gated=gated, norm=norm, pad=pad)
        self.dtype, code = TYPES[type_]
        g = torch.Generator().manual_seed(seed)
        rows = (2 if gated else 1) * I
        self.x = torch.randn((T, D), generator=g).to(self.dtype)
        self.r = (torch.randn((E, D), generator=g) * logits / math.sqrt(D)).to(self.dtype)
        w1, w2 = torch.randn((E, rows, D), generator=g) * size, torch.randn((E, D, I), generator=g) * size
        self.shape = lib.MoeShape(tokens=T, d_model=D, d_ff=I, experts=E, top_k=k, type=code,
                                  weight_type=lib.TYPE_E4M3 if fp8 else code, act=act, gated=gated,
                                  norm_topk=norm)
        if fp8:
            q1, q2 = [reference(m, 128) for m in w1], [reference(m, 128) for m in w2]
            self.s1 = torch.stack([s for _, s in q1]).cuda()
            self.s2 = torch.stack([s for _, s in q2]).cuda()

            def wide(q, s):
                f = s.double().t().repeat_interleave(128, 0)[:q.shape[0]]
                return q.double() * f.repeat_interleave(128, 1)[:, :q.shape[1]]
            self.w1, self.w2 = [wide(*p) for p in q1], [wide(*p) for p in q2]
            self.d1 = self.padded(torch.stack([q.view(torch.uint8) for q, _ in q1]), 0x7F)
            self.d2 = self.padded(torch.stack([q.view(torch.uint8) for q, _ in q2]), 0x7F)
        else:
            w1, w2 = w1.to(self.dtype), w2.to(self.dtype)
            self.s1 = self.s2 = None
            self.w1, self.w2 = list(w1.double()), list(w2.double())
            self.d1, self.d2 = self.padded(w1, float("nan")), self.padded(w2, float("nan"))

    def padded(self, w, fill):
        out = torch.full(w.shape[:-1] + (w.shape[-1] + self.pad,), fill, dtype=w.dtype)
        out[..., :w.shape[-1]] = w
        return out.cuda()

    def buffers(self):
        self.ids = torch.full((self.T, self.k), -7, dtype=torch.int32, device="cuda")
        self.w = torch.full((self.T, self.k), -7.0, device="cuda")
        self.y = torch.full((self.T, self.D + self.pad), 77.0, dtype=self.dtype, device="cuda")
        n = lib.moe_ffn_workspace(self.shape)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN of every type
        self.dx = self.padded(self.x, float("nan"))
        self.dr = self.padded(self.r, float("nan"))

    def call(self, stream=None):
        lib.moe_ffn(self.shape, self.dx, self.D + self.pad, self.dr, self.D + self.pad, self.d1,
                    self.D + self.pad, self.s1, self.d2, self.I + self.pad, self.s2, self.ids, self.w,
                    self.y, self.D + self.pad, self.ws, self.ws.numel(), stream=stream)

    def check(self):
        T, D, I, k = self.T, self.D, self.I, self.k
        x = self.x.double()
        logits = x @ self.r.double().t()
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.softmax(logits, 1).gather(1, order)
        if self.norm:
            p = p / p.sum(1, keepdim=True)
        assert torch.equal(self.ids.cpu().long(), order), "experts"
        assert ((self.w.cpu().double() - p).abs() <= 2 * U * p + 1e-45).all(), "weights"
        fin = torch.finfo(self.dtype)
        half = fin.eps / 2
        for t in range(T):
            y, err = torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
            size = torch.zeros(D, dtype=torch.float64)
            for s in range(k):
                e = int(order[t, s])
                u = self.w1[e] @ x[t]
                du = (D + blocks(D) + 24) * U * (self.w1[e].abs() @ x[t].abs())
                h = activation(u[:I], self.act)
                dh = du[:I] if self.act == 0 else 1.13 * du[:I] + 2.0 ** -21 * u[:I].abs()
                if self.gated:
                    dh = u[I:].abs() * dh + h.abs() * du[I:] + dh * du[I:]
                    h = h * u[I:]
                dh = dh + 3 * U * h.abs() + half * half * h.abs()
                if self.dtype == torch.float16:
                    dh = dh + 2.0 ** -25
                w2 = self.w2[e]
                y += p[t, s] * (w2 @ h)
                sz = p[t, s] * (w2.abs() @ h.abs())
                size += sz
                err += p[t, s] * (w2.abs() @ dh) + ((2 * I + blocks(I) + 24) * U + 2 * U) * sz
            err += k * U * size
            err += (y.abs() + err) * half + fin.smallest_normal * fin.eps
            got = self.y[t].cpu().double()
            assert (got[D:] == 77.0).all(), "written past the end"
            bad = (got[:D] - y).abs() - err
            assert got[:D].isfinite().all() and bad.max() <= 0, (t, int(bad.argmax()),
                                                                 float(bad.max()))

    def run(self):
        note("moe T %d D %d I %d E %d k %d %s fp8 %s act %d gated %d pad %d" % (
            self.T, self.D, self.I, self.E, self.k, self.dtype, self.s1 is not None, self.act,
            self.gated, self.pad))
        self.buffers()
        torch.cuda.synchronize()
        self.call()
        torch.cuda.synchronize()
        self.check()


SHAPES = [(1, 1, 1, 1, 1), (1, 64, 32, 4, 2), (1, 130, 70, 8, 3), (2, 128, 129, 3, 3),
          (4, 256, 256, 8, 2), (5, 513, 100, 60, 6), (8, 300, 1000, 16, 4), (16, 136, 64, 4, 1),
          (17, 96, 80, 5, 2), (33, 200, 144, 6, 3), (64, 160, 96, 4, 2), (64, 72, 40, 130, 8),
          (3, 1025, 385, 70, 32), (64, 64, 64, 1, 1)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,D,I,E,k", SHAPES)
def test_layer(T, D, I, E, k, fp8):
    Layer(T, D, I, E, k, "bf16", fp8, seed=1).run()
    Layer(T, D, I, E, k, "f16", fp8, act=lib.ACT_GELU_TANH, gated=False, norm=False, pad=3,
          seed=2).run()
    Layer(T, D, I, E, k, "bf16", fp8, act=lib.ACT_NONE, gated=False, pad=8, seed=3).run()
    Layer(T, D, I, E, k, "f16", fp8, act=lib.ACT_SILU, norm=False, pad=16, seed=4).run()


def test_equal_logits_go_to_the_lower_expert():
    for T, E, k in ((3, 70, 5), (20, 8, 8)):
        m = Layer(T, 64, 32, E, k, seed=5)
        m.r[:] = m.r[0].clone()             # every logit of a token the same
        m.run()
        m.r[E // 2:] *= 2                   # two groups of equals
        m.run()


def test_one_expert_takes_every_token():
    m = Layer(40, 64, 48, 8, 2, fp8=True, seed=6)
    m.x = m.x.abs()
    m.r = -m.r.abs()
    m.r[5] = 1.0
    m.run()
    assert (m.ids[:, 0] == 5).all()


def test_logits_closer_than_fp32_sums_resolve():
    """Two experts whose logits differ by 2^-30 of the sums that make them."""
    D = 1024
    m = Layer(2, D, 32, 3, 1, seed=7)
    m.x[:] = 1.0
    m.r[:] = 0.0
    m.r[:, 0], m.r[:, 1] = 2.0 ** 20, -2.0 ** 20
    m.r[1, 2:] = 2.0 ** -20
    m.r[2, 2:] = 2.0 ** -20
    m.r[2, D - 1] = 2.0 ** -19
    m.run()
    assert (m.ids == 2).all()


def test_nan_token_stays_in_its_row():
    m = Layer(4, 96, 64, 6, 2, seed=8)
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    clean, ids = m.y.clone(), m.ids.clone()
    m.dx[2, 5] = float("nan")
    m.call()
    torch.cuda.synchronize()
    assert m.y[2, :96].isnan().all() and ((m.ids >= 0) & (m.ids < 6)).all()
    assert m.ids[2].tolist() == [0, 1]
    for t in (0, 1, 3):
        assert torch.equal(m.y[t], clean[t]) and torch.equal(m.ids[t], ids[t])


@pytest.mark.parametrize("T", [1, 3, 64])
@pytest.mark.parametrize("type_,I,col", [("bf16", 45, 40), ("f16", 100, 3), ("bf16", 1000, 999)])
def test_infinite_weight_reaches_its_column_alone(T, type_, I, col):
    """h is held as two numbers, whose products with an infinite weight may differ in sign; the last
    columns of an odd row are read twice, masked, and must count once."""
    m = Layer(T, 77, I, 1, 1, type_, gated=False, act=lib.ACT_NONE, seed=13)
    h = m.x.double() @ m.w1[0][col]
    assert (h.abs() > 1e-4).all()     # (else a sign could be lost in rounding)
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    clean = m.y[:, :77].clone()
    m.d2[0, 9, col] = float("-inf")
    m.call()
    torch.cuda.synchronize()
    got = m.y[:, :77]
    assert torch.equal(got[:, 9].cpu().double(), -h.sign() * float("inf"))
    got[:, 9] = clean[:, 9]
    assert torch.equal(got, clean)


def test_binary16_inner_range_is_clamped():
    m = Layer(1, 64, 16, 1, 1, "f16", gated=False, act=lib.ACT_NONE, seed=9)
    m.x[:] = 64.0
    m.d1.fill_(32.0)        # h = 64 * 64 * 32 = 131072, clamped to 65504
    m.d2.fill_(2.0 ** -9)
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    assert (m.y == 16 * 65504 / 512).all()


def test_no_tokens():
    m = Layer(1, 8, 8, 2, 1)
    m.buffers()
    m.shape.tokens = 0
    m.call()
    torch.cuda.synchronize()
    assert (m.y == 77.0).all() and (m.ids == -7).all()


@pytest.mark.parametrize("T,E,k,fp8", [(1, 8, 2, False), (4, 16, 4, True), (40, 8, 2, True)])
def test_layer_in_a_graph_and_on_another_stream(T, E, k, fp8):
    """Replays and calls on another stream equal the eager calls, bit for bit."""
    m = Layer(T, 256, 192, E, k, fp8=fp8, seed=10)
    m.buffers()
    m.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.call()
    other = torch.cuda.Stream()
    for seed in range(3):
        m.dx[:, :256] = torch.randn((T, 256), generator=torch.Generator().manual_seed(seed)).to(
            m.dtype)
        m.call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (m.y, m.ids, m.w)]
        for again in (graph.replay, lambda: m.call(stream=other)):
            m.y.zero_()
            m.ids.zero_()
            m.w.zero_()
            m.ws.fill_(0xFF)
            torch.cuda.synchronize()
            again()
            torch.cuda.synchronize()
            for a, b in zip((m.y, m.ids, m.w), want):
                assert torch.equal(a, b)
