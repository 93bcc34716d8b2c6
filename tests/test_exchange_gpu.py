"""GPU tests of the exchange of tokens with the experts' order against its definition on the host.

The sort's whole numbers are held to equality.  With u = 2^-24 and h half a step of the type (h = u for
fp32), copies with a weight are off by at most (u + h) |w x|, sums of k slots by (k + 1) u of
sum |w||x| and h |y|, dw by (n + 16) u of sum |dy||x| with n the values that one thread adds in order."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note
from tests.test_i8_gpu import TYPES, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_destroy()


# ------------------------------------------------------------------------------------------- sort

def reference_sort(ids, experts):
    flat = ids.flatten().long()
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts)
    order = torch.sort(key, stable=True).indices
    n = int(valid.sum())
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(experts + 1))
    pos = torch.full_like(flat, -1)
    pos[order[:n]] = torch.arange(n)
    src = torch.full_like(flat, -1)
    src[:n] = order[:n]
    return offsets.int(), src.int(), pos.int()


class Sort:
    def __init__(self, ids, experts):
        self.ids, self.experts = ids, experts
        self.T, self.k = ids.shape
        self.dids = ids.cuda()
        self.offsets = torch.full((experts + 2,), -9, dtype=torch.int32, device="cuda")
        self.src = torch.full((self.T * self.k + 1,), -9, dtype=torch.int32, device="cuda")
        self.pos = torch.full((self.T * self.k + 1,), -9, dtype=torch.int32, device="cuda")
        n = lib.moe_sort_workspace(self.T, self.k, experts)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        lib.moe_sort(self.T, self.k, self.experts, self.dids, self.offsets, self.src, self.pos, self.ws,
                     self.ws.numel(), stream=stream)

    def check(self):
        offsets, src, pos = reference_sort(self.ids, self.experts)
        for got, want in ((self.offsets, offsets), (self.src, src), (self.pos, pos)):
            got = got.cpu()
            assert torch.equal(got[:-1], want) and int(got[-1]) == -9


@pytest.mark.parametrize("experts", [1, 2, 5, 64, 127, 128, 129, 1000, 1024])
@pytest.mark.parametrize("T,k", [(0, 1), (1, 1), (1, 32), (7, 3), (128, 8), (129, 8), (1025, 1), (700, 6),
                                 (4096, 8), (9001, 7)])
def test_sort(T, k, experts):
    g = torch.Generator().manual_seed(T * 31 + k * 7 + experts)
    ids = torch.randint(0, experts, (T, k), generator=g, dtype=torch.int32)
    for kind in ("all", "some", "one", "none"):
        if kind == "some" and T:   # padding, and numbers of no expert
            ids = ids.clone()
            for bad in (-1, experts, 2 ** 31 - 1, -2 ** 31):
                ids[torch.rand((T, k), generator=g) < 0.1] = bad
            ids[T // 2] = -1
        elif kind == "one":
            ids = torch.full((T, k), experts - 1, dtype=torch.int32)
        elif kind == "none":
            ids = torch.full((T, k), -1, dtype=torch.int32)
        note("moe_sort %dx%d of %d, %s" % (T, k, experts, kind))
        s = Sort(ids, experts)
        s.call()
        torch.cuda.synchronize()
        s.check()


def test_sort_many():
    """More entries than one pass of the most workgroups takes."""
    g = torch.Generator().manual_seed(2)
    for T, k, experts in ((70000, 8, 100), (300001, 2, 1024), (1 << 20, 1, 3)):
        s = Sort(torch.randint(-1, experts, (T, k), generator=g, dtype=torch.int32), experts)
        note("moe_sort %dx%d of %d" % (T, k, experts))
        s.call()
        torch.cuda.synchronize()
        s.check()


# --------------------------------------------------------------------------------- copies and sums

class Exchange:
    """pos: a random injection of the valid entries into `rows`, others -1 or past the end."""

    def __init__(self, T, k, cols, type_, rows=None, lost=0.2, weighted=True, pad=0, seed=0):
        self.__dict__.update(T=T, k=k, cols=cols, ld=max(cols, 1) + pad)
        self.dtype, self.code = TYPES[type_]
        self.half = U if type_ == "f32" else torch.finfo(self.dtype).eps / 2
        self.tiny = torch.finfo(self.dtype).smallest_normal * torch.finfo(self.dtype).eps
        self.rows = T * k + 3 if rows is None else rows
        g = torch.Generator().manual_seed(seed)
        n = T * k
        pos = torch.randperm(max(self.rows, n), generator=g)[:n]
        pos[pos >= self.rows] = -1
        if lost:
            drop = torch.rand(n, generator=g) < lost
            pos[drop] = torch.tensor([-1, self.rows, 2 ** 31 - 1, -2 ** 31])[torch.arange(int(drop.sum())) % 4]
        self.pos = pos.int().view(T, k)
        if T > 2:
            self.pos[T // 2] = -1   # a token of no expert
        self.valid = (self.pos >= 0) & (self.pos < self.rows)
        self.at = torch.where(self.valid, self.pos, 0).long()
        self.w = torch.randn((T, k), generator=g) if weighted else None
        self.tokens = torch.randn((T, cols), generator=g).to(self.dtype)
        self.sorted = torch.randn((self.rows, cols), generator=g).to(self.dtype)
        self.dpos = self.pos.cuda()
        dw = None if self.w is None else torch.where(self.valid, self.w, float("nan"))   # not read where lost
        self.dw_in = None if dw is None else dw.cuda()
        self.dtokens, self.dsorted = self.wide(self.tokens), self.wide(self.sorted)
        # A sorted row that no entry names must not count either.
        named = torch.zeros(self.rows, dtype=torch.bool)
        named[self.at[self.valid]] = True
        self.dsorted[~named.cuda()] = float("nan")
        self.named = named

    def wide(self, x):
        out = torch.full((x.shape[0], self.ld), float("nan"), dtype=x.dtype)
        out[:, :self.cols] = x
        return out.cuda()

    def blank(self, rows):
        return torch.full((rows + 1, self.ld + 1), 77.0, dtype=self.dtype, device="cuda")

    def weights(self):
        one = torch.ones((self.T, self.k)) if self.w is None else self.w
        return torch.where(self.valid, one, 0.0).double()

    def within(self, got, want, bound):
        err = (got.double() - want).abs()
        assert (err <= bound + self.tiny).all(), float((err - bound).max())

    def copies(self, got):
        """Sorted rows from tokens."""
        want = torch.full((self.rows + 1, self.ld + 1), 77.0, dtype=torch.float64)
        bound = torch.zeros_like(want)
        v = (self.weights()[..., None] * self.tokens.double()[:, None])[self.valid]
        want[self.at[self.valid], :self.cols] = v
        bound[self.at[self.valid], :self.cols] = v.abs() * (0 if self.w is None else U + self.half)
        self.within(got.cpu(), want, bound)

    def dispatch(self, stream=None):
        self.y = self.blank(self.rows)
        lib.moe_dispatch(self.T, self.k, self.cols, self.code, self.dtokens, self.ld, self.dpos, self.dw_in,
                         self.y, self.ld + 1, self.rows, stream=stream)

    def check_dispatch(self):
        self.copies(self.y)

    def combine(self, stream=None):
        self.z = self.blank(self.T)
        lib.moe_combine(self.T, self.k, self.cols, self.code, self.dsorted, self.ld, self.rows, self.dpos,
                        self.dw_in, self.z, self.ld + 1, stream=stream)

    def check_combine(self):
        w, x = self.weights()[..., None], self.sorted.double()[self.at] if self.rows else 0.0
        want = torch.full((self.T + 1, self.ld + 1), 77.0, dtype=torch.float64)
        bound = torch.zeros_like(want)
        if self.T and self.cols:
            y, size = (w * x).sum(1), (w * x).abs().sum(1)
            want[:self.T, :self.cols] = y
            bound[:self.T, :self.cols] = (self.k + 1) * U * size + self.half * (y.abs() + self.k * U * size)
        self.within(self.z.cpu(), want, bound)

    def grad(self, dx=True, dw=True, stream=None):
        self.gx = self.blank(self.rows) if dx else None
        self.gw = torch.full((self.T * self.k + 1,), 77.0, device="cuda") if dw else None
        lib.moe_combine_grad(self.T, self.k, self.cols, self.code, self.dtokens, self.ld,
                             self.dsorted if dw else None, self.ld, self.rows, self.dpos, self.dw_in,
                             self.gx, self.ld + 1, self.gw, stream=stream)

    def check_grad(self):
        if self.gx is not None:
            self.copies(self.gx)
        if self.gw is not None:
            x = self.sorted.double()[self.at] if self.rows else torch.zeros((self.T, self.k, self.cols))
            prod = torch.where(self.valid[..., None], self.tokens.double()[:, None] * x, 0.0)
            n = 8 * (-(-self.cols // 1024)) + 16
            got = self.gw.cpu().double()
            assert float(got[-1]) == 77.0
            err = (got[:-1].view(self.T, self.k) - prod.sum(2)).abs()
            assert (err <= n * U * prod.abs().sum(2)).all()
            assert (got[:-1].view(self.T, self.k)[~self.valid] == 0).all()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("T,k,cols", [(1, 1, 1), (3, 2, 3), (5, 1, 4), (4, 3, 7), (9, 2, 8), (6, 8, 9),
                                      (40, 6, 100), (33, 9, 255), (17, 17, 513), (5, 32, 1000),
                                      (300, 8, 2050), (7, 4, 5000), (2, 5, 20001)])
def test_exchange(T, k, cols, type_):
    for weighted, pad in ((True, 0), (False, 3)):
        e = Exchange(T, k, cols, type_, weighted=weighted, pad=pad, seed=T + k + cols)
        note("exchange %dx%d cols %d %s weighted %s" % (T, k, cols, type_, weighted))
        e.dispatch()
        e.combine()
        torch.cuda.synchronize()
        e.check_dispatch()
        e.check_combine()
        for dx, dw in ((True, True), (True, False), (False, True)):
            e.grad(dx, dw)
            torch.cuda.synchronize()
            e.check_grad()


def test_few_rows_and_none():
    """Fewer sorted rows than entries; no rows, no columns."""
    for T, k, cols, rows in ((20, 3, 50, 17), (20, 3, 50, 0), (20, 3, 0, 60), (0, 3, 50, 5)):
        e = Exchange(T, k, cols, "bf16", rows=rows, lost=0.0)
        note("exchange %dx%d cols %d rows %d" % (T, k, cols, rows))
        e.dispatch()
        e.combine()
        e.grad()
        torch.cuda.synchronize()
        e.check_dispatch()
        e.check_combine()
        e.check_grad()


def test_rows_past_4_gib():
    """Sorted rows and tokens whose bytes begin past 2^32."""
    T, cols = 9, 1 << 20
    rows = 2 ** 32 // (2 * cols) + 20
    tokens = torch.randn((T, cols), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pos = torch.arange(rows - T, rows, dtype=torch.int32, device="cuda")
    y = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    note("exchange past 4 GiB")
    lib.moe_dispatch(T, 1, cols, lib.TYPE_BF16, tokens, cols, pos, None, y, cols, rows)
    back = torch.empty_like(tokens)
    lib.moe_combine(T, 1, cols, lib.TYPE_BF16, y, cols, rows, pos, None, back, cols)
    assert torch.equal(y[rows - T:], tokens) and not y[:rows - T].any()
    assert torch.equal(back, tokens)


def test_gradients_against_differences():
    """The loss sum(G * Y) is linear in every value that the gradients are for: a difference over any step
    is the gradient, up to the rounding of the sums that are subtracted."""
    e = Exchange(12, 3, 40, "f32", lost=0.1, seed=5)
    g = torch.randn((e.T, e.cols), generator=torch.Generator().manual_seed(6))

    def loss():
        e.combine()
        return float((e.z[:e.T, :e.cols].cpu().double() * g.double()).sum())
    keep = e.dtokens
    e.dtokens = e.wide(g)
    e.grad()
    gx, gw = e.gx.cpu(), e.gw.cpu()
    e.dtokens = keep
    w, x = e.dw_in.clone(), e.dsorted.clone()
    size = float((e.weights()[..., None] * e.sorted.double()[e.at] * g.double()[:, None]).abs().sum())
    tol = 2 * 8 * U * (size + 100)
    for t, s in ((0, 0), (3, 2), (6, 1), (11, 1)):
        if e.valid[t, s]:
            up, down = w.clone(), w.clone()
            up[t, s] += 1
            down[t, s] -= 1
            e.dw_in = up
            high = loss()
            e.dw_in = down
            assert abs((high - loss()) / 2 - float(gw[t * e.k + s])) <= tol
            e.dw_in = w
            row, col = int(e.pos[t, s]), 7 * s
            high = e.dsorted[row, col] = x[row, col] + 1
            high = loss()
            e.dsorted[row, col] = x[row, col] - 1
            assert abs((high - loss()) / 2 - float(gx[row, col])) <= tol
            e.dsorted[row, col] = x[row, col]


def test_dispatch_gradients_are_the_documented_calls():
    """To X: combine of Y's gradient; to w: combine_grad's dw with the two exchanged."""
    e = Exchange(30, 4, 70, "f32", lost=0.1, seed=8)
    tokens, rows = e.tokens.double().requires_grad_(), e.sorted.double()
    w = e.weights().requires_grad_()
    y = (w[..., None] * tokens[:, None])[e.valid]
    (y * rows[e.at[e.valid]]).sum().backward()   # e.sorted plays Y's gradient
    e.combine()
    e.grad(dx=False)
    got = e.z[:e.T, :e.cols].cpu().double()
    size = (e.weights()[..., None] * rows[e.at]).abs().sum(1)
    assert ((got - tokens.grad).abs() <= (e.k + 2) * U * size).all()
    want = torch.where(e.valid, w.grad, 0.0)
    size = (e.tokens.double()[:, None] * rows[e.at]).abs().sum(2)
    assert ((e.gw[:-1].cpu().double().view(e.T, e.k) - want).abs() <= 24 * U * size).all()


def test_streams_and_graph():
    s, e = Sort(torch.randint(-1, 16, (300, 6), dtype=torch.int32), 16), Exchange(50, 4, 300, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.call()
        e.dispatch()
        e.combine()
        e.grad()
    torch.cuda.synchronize()
    s.check()
    e.check_dispatch()
    e.check_combine()
    e.check_grad()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call()
        e.dispatch()
        e.combine()
        e.grad()
    for i in range(3):
        s.ids = torch.randint(-1, 16, (300, 6), generator=torch.Generator().manual_seed(i), dtype=torch.int32)
        s.dids.copy_(s.ids)
        e.tokens = torch.randn(e.tokens.shape, generator=torch.Generator().manual_seed(i)).to(e.dtype)
        e.dtokens[:, :e.cols] = e.tokens.cuda()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check()
        e.check_dispatch()
        e.check_combine()
        e.check_grad()
