"""GPU tests of the row quantisation to int8 and of the int8 product, plain and grouped, against their
definitions.

Quantised values and scales are held to equality with the definition in fp32 (torch's division on the
CPU rounds to nearest, as IEEE asks).  The product's sums are exact; with u = 2^-24 its result is
off by at most
  scaled   - 3 u |sa sb sum| (the sum, the scales' product, theirs) and a 4th u for what that leaves out,
             times |alpha|, and u of the value with its bias;
  act      - a slope of at most 1.13 and 2^-21 |x| of its own;
  gate     - |act| dv + |v| dact + both, and u;
  result   - half a step of its type."""
import math

import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": (torch.float32, lib.TYPE_F32), "f16": (torch.float16, lib.TYPE_F16),
         "bf16": (torch.bfloat16, lib.TYPE_BF16)}


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_debug_force_i8_tile(-1)
    lib.gemm_destroy()


# ------------------------------------------------------------------------------------ quantisation

def reference_rows(x):
    """Q and S of rows, by the definition (host)."""
    x = x.float()
    m = x.abs().amax(1)
    s = m / torch.tensor(127.0)
    s = torch.where(s < 2.0 ** -126, torch.tensor(2.0 ** -126), s)   # (NaN stays)
    q = torch.round(x / s[:, None])
    q = torch.where(torch.isfinite(s)[:, None], q, torch.tensor(0.0))
    return q.to(torch.int8), s


def check_rows(x, pad=0, offset=0):
    rows, cols = x.shape
    code = [c for t, c in TYPES.values() if t == x.dtype][0]
    want_q, want_s = reference_rows(x)
    dx = torch.full((rows * (cols + pad) + offset,), float("nan"), dtype=x.dtype)
    dx[offset:].view(rows, cols + pad)[:, :cols] = x
    dx = dx.cuda()
    q = torch.full((rows, cols + pad + 3), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), -7.0, device="cuda")
    note("i8_quantize %dx%d %s pad %d" % (rows, cols, x.dtype, pad))
    lib.i8_quantize(rows, cols, code, dx[offset:], cols + pad, q, cols + pad + 3, s)
    torch.cuda.synchronize()
    s, q = s.cpu(), q.cpu()
    assert float(s[rows]) == -7.0 and (q[:, cols:] == 77).all(), "written past the end"
    assert torch.equal(torch.nan_to_num(s[:rows], -1.0), torch.nan_to_num(want_s, -1.0)), "scales"
    assert torch.equal(q[:, :cols], want_q), "values"


def spread(g, rows, cols):
    return torch.randn((rows, cols), generator=g) * torch.exp(2 * torch.randn((rows, 1), generator=g))


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (5, 7), (2, 8), (9, 9), (3, 64), (300, 100),
                                       (1, 513), (8, 4096), (2100, 520), (5, 4100), (2100, 4096),
                                       (7, 14336), (3, 16385), (2, 40001), (2, 70001), (1, 1 << 20)])
def test_rows(type_, rows, cols):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = spread(g, rows, cols).to(TYPES[type_][0])
    check_rows(x)
    if rows * cols < 1 << 18:
        check_rows(x, pad=5, offset=1)


@pytest.mark.parametrize("type_", list(TYPES))
def test_special_rows(type_):
    """Zeros, NaN, infinities, the smallest and largest numbers, in rows of one and of many waves."""
    fin = torch.finfo(TYPES[type_][0])
    tiny = fin.smallest_normal * fin.eps   # the smallest subnormal
    for cols in (4, 100, 3000, 30000, 70000):
        x = torch.randn((12, cols), generator=torch.Generator().manual_seed(cols))
        x[0] = 0
        x[1, cols - 1] = float("nan")
        x[2, 0] = float("inf")
        x[3, cols // 2] = float("-inf")
        x[4, 0], x[4, 3] = float("nan"), float("inf")
        x[5], x[6] = -0.0, 1.0
        x[7] = x[7].sign() * tiny
        x[8] = (x[8] * 1000).trunc() * tiny
        x[9] = x[9].sign() * fin.max
        x[10] = x[10] * fin.smallest_normal
        x[11] = x[11] * 2.0 ** -62 if type_ != "f16" else x[11] * 2.0 ** -20
        check_rows(x.to(TYPES[type_][0]))


def test_ties():
    """Every whole number and a half of a row whose scale is a power of two: ties go to even."""
    x = torch.arange(-127, 127.5, 0.5)[None] * torch.exp2(torch.arange(-100, 100, 7.0))[:, None]
    check_rows(x)
    check_rows(x.to(torch.bfloat16)[:, ::2])


def test_many_quotients():
    """About 4 million bfloat16 quotients with 1024 scales."""
    x = torch.randn((1024, 4096), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    check_rows(x)


# ---------------------------------------------------------------------------------------- product

def activation(x, act):
    if act == lib.ACT_GELU_TANH:
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x / (1 + torch.exp(-x)) if act == lib.ACT_SILU else x


def reference_product(a, sa, b, sb, alpha, bias, act, gated, dtype):
    """(C, its bound) of a group's rows in 64 bits; a, b int8 (host)."""
    acc = a.double() @ b.double().t()
    x = alpha * (sa.double()[:, None] * sb.double() * acc)
    dx = 4 * U * x.abs()
    if bias is not None:
        x = x + bias.double()
    dx = dx + U * x.abs()
    n = b.shape[0] // 2 if gated else b.shape[0]
    y = activation(x[:, :n], act)
    dy = dx[:, :n] if act == 0 else 1.13 * dx[:, :n] + 2.0 ** -21 * x[:, :n].abs()
    if gated:
        v, dv = x[:, n:], dx[:, n:]
        dy = y.abs() * dv + v.abs() * dy + dy * dv
        y = y * v
        dy = dy + U * y.abs()
    fin = torch.finfo(dtype)
    if dtype != torch.float32:
        dy = dy + (y.abs() + dy) * fin.eps / 2
    return y, dy + fin.smallest_normal * fin.eps


def int8s(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def scales(g, n, size):
    return torch.exp(torch.randn(n, generator=g)) * size


def padded(x, ld, fill=-128):
    out = torch.full(x.shape[:-1] + (ld,), fill, dtype=x.dtype)
    out[..., :x.shape[-1]] = x
    return out.cuda()


class Product:
    """Operands of a product or, with `rows` (of every group), of a grouped one."""

    def __init__(self, M, N, K, type_="bf16", bias=True, act=0, gated=False, alpha=1.0, pad=0, seed=0,
                 rows=None, first=0, gather=None, per=1, off=0):
        self.__dict__.update(M=M, N=N, K=K, act=act, gated=gated, alpha=alpha, per=per, rows=rows)
        self.dtype, self.code = TYPES[type_]
        g = torch.Generator().manual_seed(seed)
        groups = 1 if rows is None else len(rows)
        self.a_rows = M if gather is None else gather
        self.a, self.sa = int8s(g, self.a_rows, K), scales(g, self.a_rows, 0.01)
        wide = N * (1 + gated)
        self.b, self.sb = int8s(g, groups, wide, K), scales(g, groups * wide, 0.003).view(groups, wide)
        self.bias = torch.randn((groups, wide), generator=g) if bias else None
        self.ld = -(-K // 16) * 16 if pad else max(K, 1)

        def at(x):   # `off` bytes behind a 16-byte boundary
            d = torch.full((x.numel() + 16,), -128, dtype=torch.int8, device="cuda")
            d[off:off + x.numel()] = x.flatten()
            return d[off:]
        self.da, self.db = at(padded(self.a, self.ld)), at(padded(self.b, self.ld))
        self.dsa, self.dsb = self.sa.cuda(), self.sb.cuda()
        self.dbias = None if self.bias is None else self.bias.cuda()
        self.ldc = N + 3
        self.c = torch.full((M + 1, self.ldc), 77.0, dtype=self.dtype, device="cuda")
        self.index = self.dindex = None
        if rows is not None:
            self.offsets = torch.tensor([first] + [first + sum(rows[:i + 1]) for i in range(groups)],
                                        dtype=torch.int32)
            assert int(self.offsets[-1]) <= M
            self.doffsets = self.offsets.cuda()
            if gather is not None:
                self.index = torch.randint(0, gather * per, (M,), generator=g, dtype=torch.int32)
                self.dindex = self.index.cuda()

    def call(self, stream=None):
        tail = (self.dbias, self.act, self.gated, self.code, self.c, self.ldc)
        if self.rows is None:
            lib.i8_gemm_bias_act(self.M, self.N, self.K, self.alpha, self.da, self.ld, self.dsa, self.db,
                                 self.ld, self.dsb, *tail, stream=stream)
        else:
            lib.i8_gemm_grouped(len(self.rows), self.doffsets, self.M, self.N, self.K, self.alpha, self.da,
                                self.ld, self.dsa, self.a_rows, self.dindex, self.per, self.db, self.ld,
                                self.dsb, *tail, stream=stream)

    def check(self):
        got = self.c.cpu()
        want = torch.full(got.shape, 77.0, dtype=torch.float64)
        bound = torch.zeros_like(want)
        for g in range(self.b.shape[0]):
            lo, hi = (0, self.M) if self.rows is None else self.offsets[g:g + 2].tolist()
            if lo == hi or self.N == 0:
                continue
            read = torch.arange(lo, hi) if self.index is None else self.index[lo:hi].long() // self.per
            y, dy = reference_product(self.a[read], self.sa[read], self.b[g], self.sb[g], self.alpha,
                                      None if self.bias is None else self.bias[g], self.act, self.gated,
                                      self.dtype)
            want[lo:hi, :self.N], bound[lo:hi, :self.N] = y, dy
        err = (got.double() - want).abs()
        # From half a step past the type's largest number on, the nearest one is infinite.
        fin = torch.finfo(self.dtype)
        past = (want.abs() + bound >= fin.max * (1 + fin.eps / 4)) & (got.double() == want.sign() * math.inf)
        assert ((err <= bound) | past).all(), "worst %g of its bound at %s" % (
            float((err / bound.clamp_min(1e-300))[~past].max()),
            divmod(int(torch.where(past, 0.0, err - bound).argmax()), self.ldc))


def run(p, tile=-1):
    lib.gemm_debug_force_i8_tile(tile)
    p.call()
    torch.cuda.synchronize()
    p.check()
    lib.gemm_debug_force_i8_tile(-1)


OPTIONS = [dict(), dict(type_="f32", act=2, gated=True), dict(type_="f16", act=1, bias=False, alpha=0.5),
           dict(act=1, gated=True, bias=False), dict(type_="f32", act=0, alpha=-2.0),
           dict(type_="f16", act=0, gated=True, alpha=1.5), dict(act=2, bias=False)]


@pytest.mark.parametrize("tile", range(-1, 12))
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 300, 128), (17, 33, 100), (64, 64, 64), (130, 250, 129),
                                   (33, 70, 1040), (257, 140, 2064), (300, 520, 777)])
def test_product(M, N, K, tile):
    n = M + N + K + tile
    for pad, off in ((1, 0), (0, 0), (1, 5)):
        option = OPTIONS[(n + pad + off) % len(OPTIONS)]
        note("i8 product %dx%dx%d tile %d pad %d off %d %s" % (M, N, K, tile, pad, off, option))
        run(Product(M, N, K, pad=pad, off=off, seed=n, **option), tile)


@pytest.mark.parametrize("option", OPTIONS)
@pytest.mark.parametrize("tile", range(-1, 12))
def test_options(option, tile):
    note("i8 product options tile %d %s" % (tile, option))
    run(Product(70, 90, 400, pad=1, seed=3, **option), tile)


@pytest.mark.parametrize("tile", [-1, 0, 1, 2, 4, 5, 6, 7, 11])
def test_nothing_to_sum(tile):
    for K, alpha in ((0, 1.0), (40, 0.0)):
        note("i8 product K %d alpha %g tile %d" % (K, alpha, tile))
        p = Product(20, 35, K, alpha=alpha, act=1, type_="f32")
        if alpha == 0.0:
            p.dsa.fill_(float("nan"))   # not read
            p.sa, p.a = torch.ones(20), torch.zeros_like(p.a)
        run(p, tile)
    p = Product(0, 35, 64)
    run(p, tile)


@pytest.mark.parametrize("tile", [-1, 0, 1, 2, 4, 5, 6, 7, 11])
def test_longest_sums(tile):
    """131071 products of -128 and -128: 2^31 - 2^14 fits int32."""
    p = Product(3, 20, 131071, pad=1, type_="f32")
    p.a.fill_(-128)
    p.b.fill_(-128)
    p.b[0, 1::2] = 127
    p.da, p.db = padded(p.a, p.ld), padded(p.b, p.ld)
    note("i8 product K 131071 tile %d" % tile)
    run(p, tile)


@pytest.mark.parametrize("tile", [-1, 0, 1, 2, 4, 5, 6, 7, 11])
def test_far_scales(tile):
    """Scales whose product with the sum stays in range though other orders of multiplying would not."""
    for ea, eb in ((110, -120), (-126, 100), (-126, 0), (120, -126), (-140, 100), (40, 60)):
        p = Product(9, 40, 200, pad=1, type_="f32", bias=False)
        p.sa, p.sb = torch.full((9,), 2.0 ** ea * 1.25), torch.full((1, 40), 2.0 ** eb * 1.5)
        p.dsa, p.dsb = p.sa.cuda(), p.sb.cuda()
        note("i8 product scales 2^%d 2^%d tile %d" % (ea, eb, tile))
        run(p, tile)


@pytest.mark.parametrize("tile", [-1, 0, 1, 2, 4, 5, 6, 7, 11])
def test_nan_scales(tile):
    p = Product(9, 40, 200, pad=1, type_="f32")
    for value in (float("nan"), float("inf")):
        sa = p.sa.clone()
        sa[3] = value
        p.a[3] = 0   # what the quantisation gives such a row
        p.da, p.dsa = padded(p.a, p.ld), sa.cuda()
        lib.gemm_debug_force_i8_tile(tile)
        p.call()
        torch.cuda.synchronize()
        lib.gemm_debug_force_i8_tile(-1)
        c = p.c.cpu()
        assert torch.isnan(c[3, :40]).all() and torch.isfinite(c[[0, 1, 2, 4, 5, 6, 7, 8]]).all()


GROUPS = [
    dict(M=40, rows=[3, 0, 17, 1, 0, 0, 12], first=0),
    dict(M=600, rows=[0, 130, 257, 0, 64, 1, 2], first=5),
    dict(M=8, rows=[1] * 8),
    dict(M=30, rows=[0, 0, 0]),
    dict(M=300, rows=[i % 3 for i in range(200)], first=1),
    dict(M=900, rows=[(7 * i) % 2 for i in range(1024)], first=0),
    dict(M=513, rows=[513]),
]


@pytest.mark.parametrize("tile", range(-1, 12))
@pytest.mark.parametrize("case", GROUPS, ids=lambda c: "%d-%d" % (c["M"], len(c["rows"])))
def test_grouped(case, tile):
    n = case["M"] + tile
    few = len(case["rows"]) > 100
    for i, (gather, per, pad, off) in enumerate(((None, 1, 1, 0), (11, 4, 1, 0), (50, 1, 0, 3))):
        option = OPTIONS[(n + i) % len(OPTIONS)]
        N, K = (20, 48) if few else (150, 272 + 40 * i)
        note("i8 grouped %s tile %d gather %s %s" % (case["M"], tile, gather, option))
        run(Product(N=N, K=K, gather=gather, per=per, pad=pad, off=off, seed=n, **case, **option), tile)


def test_bad_offsets_and_rows_stay_inside():
    """What the documentation leaves unspecified may come out anyhow, but only inside the arrays."""
    for tile in range(-1, 12):
        p = Product(40, 50, 100, rows=[10, 10, 10, 10], gather=7, per=2, pad=1)
        p.doffsets = torch.tensor([-5, 30, 12, 100000, 20], dtype=torch.int32, device="cuda")
        p.dindex = torch.tensor([-7, 2 ** 31 - 1, 3, -2 ** 31, 900] * 8, dtype=torch.int32, device="cuda")
        note("i8 grouped bad offsets tile %d" % tile)
        lib.gemm_debug_force_i8_tile(tile)
        p.call()
        torch.cuda.synchronize()
        lib.gemm_debug_force_i8_tile(-1)
        c = p.c.cpu()
        assert (c[40] == 77.0).all() and (c[:, 50:] == 77.0).all()


@pytest.mark.parametrize("tile", [-1, 0, 1, 3, 5, 8, 11])
def test_matrices_past_4_gib(tile):
    """The last group's matrix begins past 2^32 bytes; with an index so do rows of A."""
    groups, N, K = 9, 32768, 16384
    g = torch.Generator().manual_seed(1)
    b = torch.zeros((groups, N, K), dtype=torch.int8, device="cuda")
    last = int8s(g, N, K)
    b[groups - 1] = last.cuda()
    a = torch.zeros((2 ** 32 // K + 5, K), dtype=torch.int8, device="cuda")
    tail = int8s(g, 3, K)
    a[-3:] = tail.cuda()
    sa, sb = torch.ones(a.shape[0], device="cuda"), torch.ones((groups, N), device="cuda")
    index = torch.tensor([a.shape[0] - 3, a.shape[0] - 1, a.shape[0] - 2], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0] * groups + [3], dtype=torch.int32, device="cuda")
    want = (tail.double()[[0, 2, 1]] @ last[-40:].double().t()).float()
    for rows, x in ((a.shape[0], index), (3, None)):
        c = torch.zeros((3, N), device="cuda")
        note("i8 grouped past 4 GiB tile %d rows %d" % (tile, rows))
        lib.gemm_debug_force_i8_tile(tile)
        lib.i8_gemm_grouped(groups, offsets, 3, N, K, 1.0, a if x is not None else a[-3:][[0, 2, 1]].contiguous(),
                            K, sa, rows, x, 1, b, K, sb, None, 0, False, lib.TYPE_F32, c, N)
        torch.cuda.synchronize()
        lib.gemm_debug_force_i8_tile(-1)
        assert torch.equal(c[:, -40:].cpu(), want)


@pytest.mark.parametrize("tile", [-1, 0, 1, 2, 3, 4, 5, 8])
def test_offsets_between_2_and_4_gib(tile):
    """Rows of A read by index, and the second half of a gated B, begin past 2^31 bytes of the first."""
    N, K, rows = 140000, 16384, 3 * 2 ** 30 // 16384
    g = torch.Generator().manual_seed(2)
    a = torch.zeros((rows, K), dtype=torch.int8, device="cuda")
    tail = int8s(g, 2, K)
    a[-2:] = tail.cuda()
    b = torch.zeros((2 * N, K), dtype=torch.int8, device="cuda")
    last = int8s(g, 2, 40, K)
    b[N - 40:N], b[2 * N - 40:] = last[0].cuda(), last[1].cuda()
    sa, sb = torch.ones(rows, device="cuda"), torch.full((2 * N,), 2.0 ** -10, device="cuda")
    index = torch.tensor([rows - 1, rows - 2], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    c = torch.zeros((2, N), device="cuda")
    note("i8 grouped between 2 and 4 GiB tile %d" % tile)
    lib.gemm_debug_force_i8_tile(tile)
    lib.i8_gemm_grouped(1, offsets, 2, N, K, 1.0, a, K, sa, rows, index, 1, b, K, sb, None, 0, True,
                        lib.TYPE_F32, c, N)
    torch.cuda.synchronize()
    lib.gemm_debug_force_i8_tile(-1)
    x, one = tail[[1, 0]], torch.ones(2)
    y, bound = reference_product(x, one, last.view(80, K), torch.full((80,), 2.0 ** -10), 1.0, None, 0, True,
                                 torch.float32)
    assert ((c[:, -40:].cpu().double() - y).abs() <= bound).all() and not c[:, :-40].any()


@pytest.mark.parametrize("rows", [None, [5, 0, 27, 1]])
def test_weights_larger_than_the_caches(rows):
    """About 100 MB of weights for few rows: copied past the caches."""
    M, N = (31, 6001) if rows is None else (40, 1501)
    p = Product(M, N, 8208, pad=1, gated=True, act=2, type_="f32", rows=rows, first=0)
    assert p.b.numel() >= 96e6
    for tile in range(-1, 6):
        note("i8 product of 100 MB of weights, tile %d, rows %s" % (tile, rows))
        p.c.fill_(77.0)
        run(p, tile)


def test_random_shapes():
    g = torch.Generator().manual_seed(11)
    for i in range(30):
        M, N, K = (int(2 ** (8.5 * torch.rand(1, generator=g))) for _ in range(3))
        p = Product(M, N, 4 * K + i % 5, pad=i % 3, seed=i, **OPTIONS[i % len(OPTIONS)])
        note("i8 random %d: %dx%dx%d" % (i, M, N, 4 * K + i % 5))
        run(p)


def test_streams_and_graph():
    p, q = Product(70, 300, 520, pad=1), Product(300, 90, 256, rows=[100, 0, 150, 20], gather=40, per=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.call(stream=side)
    with torch.cuda.stream(side):
        q.call()
    torch.cuda.synchronize()
    p.check()
    q.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call()
        q.call()
    for i in range(3):
        p.a, p.c[:] = int8s(torch.Generator().manual_seed(i), *p.a.shape), 77.0
        p.da[:p.a.shape[0] * p.ld].view(-1, p.ld)[:, :p.K] = p.a.cuda()
        q.rows = [50 + i, 3, 0, 200]
        q.offsets = torch.tensor([0, 50 + i, 53 + i, 53 + i, 253 + i], dtype=torch.int32)
        q.doffsets.copy_(q.offsets)
        q.c[:] = 77.0
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p.check()
        q.check()
