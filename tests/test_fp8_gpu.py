"""GPU tests of block quantisation and the block-scaled e4m3 product against their definitions.

Quantisation is held to equality: scale and quotient are correctly rounded divisions, in fp32 for
16-bit values and in 64 bits for fp32 ones, which the CPU forms too.  The product is held to a bound
of its own roundings, with u = 2^-24:
  exact sums  - a block's 128 exact products are added in fp32 (at most 128 roundings), each block's
                sum meets two roundings of its scale and one of its addition, eight partial totals are
                added: (128 + blocks + 16) u of sum |s_a a s_b b|;
  fast sums   - 2^-11 of the same sum (twice the largest error measured of the instruction's adder);
  activation  - a slope of at most 1.13, and 2^-21 |x| from the exponential and the reciprocal;
  result      - half a step of its type."""
import pytest
import torch

import linear_algebra_sgemm_amd as lib
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": (torch.float32, lib.TYPE_F32), "f16": (torch.float16, lib.TYPE_F16),
         "bf16": (torch.bfloat16, lib.TYPE_BF16)}
E4M3 = torch.float8_e4m3fn
SENTINEL = 0x55


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib.gemm_create()
    yield
    torch.cuda.synchronize()
    lib.gemm_destroy()


def blocks(n, of=128):
    return -(-n // of)


def reference(x, b):
    """Scales (blocks of columns first) and e4m3 values of a CPU matrix: scale and quotient in fp32
    for 16-bit values, for fp32 ones in 64 bits."""
    rows, cols = x.shape
    wide = torch.float64 if x.dtype == torch.float32 else torch.float32
    y = torch.zeros((blocks(rows, b) * b, blocks(cols) * 128), dtype=wide)
    y[:rows, :cols] = x.to(wide)
    y = y.reshape(blocks(rows, b), b, blocks(cols), 128)
    amax = y.abs().amax(dim=(1, 3))
    s = (amax * (1.0 / 448) if wide == torch.float64 else amax / 448).clamp_min(2.0 ** -126)
    q = (y / s[:, None, :, None]).reshape(blocks(rows, b) * b, -1)[:rows, :cols].double()
    # Nearest multiple of e4m3's spacing at the value's size, ties to even.
    space = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / space) * space).float().to(E4M3), s.float().t().contiguous()


def run_quantize(x, b, plain=True, turned=True, pad=0, offset=0):
    """x: CPU matrix.  Outputs with `pad` more columns, which must stay as they were."""
    rows, cols = x.shape
    type_ = [c for t, c in TYPES.values() if t == x.dtype][0]
    ldx = cols + pad
    d = torch.full((rows * ldx + offset,), float("nan"), dtype=x.dtype, device="cuda")
    X = d[offset:].view(rows, ldx)
    X[:, :cols] = x.cuda()
    out = []
    for wanted, (r, c) in ((plain, (rows, cols)), (turned, (cols, rows))):
        if wanted:
            Q = torch.full((r * (c + pad) + offset,), SENTINEL, dtype=torch.uint8, device="cuda")
            S = torch.full((blocks(c), (r if b == 1 else blocks(r)) + pad), -1.0, device="cuda")
            out.append((Q, S, r, c))
        else:
            out.append(None)
    args = []
    for o in out:
        args += [None, 0, None, 0] if o is None else [o[0].data_ptr() + offset, o[3] + pad, o[1],
                                                      o[1].shape[1]]
    lib.fp8_quantize(rows, cols, type_, X, ldx, b, *args)
    torch.cuda.synchronize()
    got = []
    for o in out:
        if o is None:
            got.append(None)
            continue
        Q, S, r, c = o
        Q = Q.cpu()
        assert (Q[:offset] == SENTINEL).all()
        Q, S = Q[offset:].view(r, c + pad), S.cpu()
        n = r if b == 1 else blocks(r)
        assert (Q[:, c:] == SENTINEL).all() and (S[:, n:] == -1).all(), "written past the end"
        got.append((Q[:, :c].contiguous(), S[:, :n]))
    return got


def check_quantize(x, b, **kw):
    plain, turned = run_quantize(x, b, **kw)
    for got, m in ((plain, x), (turned, x.t())):
        if got is None:
            continue
        q, s = reference(m, b)
        gq, gs = got[0].view(E4M3).float(), got[1]
        assert torch.equal(gs.isnan(), s.isnan()) and torch.equal(gs.nan_to_num(3), s.nan_to_num(3))
        assert torch.equal(gq.isnan(), q.float().isnan())
        assert torch.equal(gq.nan_to_num(7), q.float().nan_to_num(7))


def matrix(rows, cols, type_, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(torch.randn((rows, 1), generator=g))
    x *= 1 + 30 * (torch.rand((1, cols), generator=g) < 0.02)
    return x.to(TYPES[type_][0])


@pytest.mark.parametrize("type_", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (128, 1), (7, 129), (128, 128), (129, 127),
                                       (64, 256), (300, 520), (1000, 64), (17, 1001)])
def test_quantize(rows, cols, b, type_):
    note("quantize %dx%d block %d %s" % (rows, cols, b, type_))
    x = matrix(rows, cols, type_, rows + cols)
    check_quantize(x, b)
    check_quantize(x, b, turned=False, pad=3, offset=1)
    check_quantize(x, b, plain=False, pad=5, offset=3)
    check_quantize(x, b, pad=8, offset=8)


@pytest.mark.parametrize("type_", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b", [1, 128])
def test_quantize_special_values(b, type_):
    x = matrix(260, 390, type_, 5)
    x[3, 5] = float("nan")
    x[140, 140] = float("inf")
    x[200, 300] = float("-inf")
    x[10:20] = 0
    x[:, 50:60] = 0
    x[128:256, 256:384] = 0           # a whole block of zeros
    tiny = torch.finfo(x.dtype).tiny
    x[30] = tiny / 4                  # subnormal numbers
    x[31, ::2] = -0.0
    x[40] = torch.finfo(x.dtype).max
    x[41] = -torch.finfo(x.dtype).max
    note("quantize special values block %d %s" % (b, type_))
    check_quantize(x, b)
    check_quantize(x, b, turned=False)


@pytest.mark.parametrize("b", [1, 128])
def test_quantize_ties(b):
    # Multiples of 1/2 of e4m3's spacing at amax = 448: scale 1, so every tie is exact.
    steps = torch.arange(1, 897) / 2.0
    x = torch.zeros((128, 128 * 7))
    x[:, :] = steps[None, :896]
    x[:, ::128] = 448
    check_quantize(x, b)
    check_quantize(-x, b)


def test_quantize_empty_and_stream():
    e = torch.empty((0, 5), dtype=torch.bfloat16, device="cuda")
    lib.fp8_quantize(0, 5, lib.TYPE_BF16, e, 5, 1, e, 5, torch.empty(1, device="cuda"), 1)
    s = torch.cuda.Stream()
    x = matrix(256, 256, "bf16", 3)
    d, Q, S = x.cuda(), torch.empty((256, 256), dtype=torch.uint8, device="cuda"), torch.empty(
        (2, 256), device="cuda")
    torch.cuda.synchronize()
    lib.fp8_quantize(256, 256, lib.TYPE_BF16, d, 256, 1, Q, 256, S, 256, stream=s)
    s.synchronize()
    q, sc = reference(x, 1)
    assert torch.equal(Q.cpu(), q.view(torch.uint8)) and torch.equal(S.cpu(), sc)


# --------------------------------------------------------------------------------------- the product

def activation(x, act):
    if act == lib.ACT_GELU_TANH:
        return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x ** 3)))
    return x / (1 + torch.exp(-x)) if act == lib.ACT_SILU else x


def operands(M, N, K, b_rows, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def normal(r, c, size):
        x = torch.randn((r, c), generator=g) * size
        return x * torch.exp(spread * torch.randn((r, c), generator=g)) if spread != 1.0 else x
    a, sa = reference(normal(M, K, 1.0), 1)
    b, sb = reference(normal(N, K, 0.05), b_rows)
    return a, sa, b, sb


def check_product(M, N, K, type_="f32", act=0, bias=True, b_rows=128, fast=False, alpha=1.0, pad=0,
                  offset=0, seed=0, spread=1.0):
    note("fp8 product %dx%dx%d %s act %d b_rows %d fast %d pad %d" % (M, N, K, type_, act, b_rows,
                                                                     fast, pad))
    dtype, code = TYPES[type_]
    a, sa, b, sb = operands(M, N, K, b_rows, seed, spread)
    g = torch.Generator().manual_seed(seed + 1)
    bv = torch.randn((N,), generator=g) if bias else None

    def padded(q):   # rows of K + pad bytes, the pad NaN
        d = torch.full((q.shape[0] * (K + pad) + offset,), 0x7F, dtype=torch.uint8, device="cuda")
        d[offset:].view(q.shape[0], K + pad)[:, :K] = q.view(torch.uint8).cuda()
        return d
    def scales(x):   # rows of 3 more values where the matrices are padded, NaN too
        d = torch.full((x.shape[0], x.shape[1] + (3 if pad else 0)), float("nan"))
        d[:, :x.shape[1]] = x
        return d.cuda()
    dA, dB, dSA, dSB = padded(a), padded(b), scales(sa), scales(sb)
    ldc = N + pad
    C = torch.full((M, ldc), 77.0, dtype=dtype, device="cuda")
    lib.fp8_gemm_bias_act(M, N, K, alpha, dA.data_ptr() + offset, K + pad, dSA, dSA.shape[1],
                          dB.data_ptr() + offset, K + pad, dSB, dSB.shape[1], b_rows,
                          None if bv is None else bv.cuda(), act, code, C, ldc, fast_sums=fast)
    torch.cuda.synchronize()
    got = C.cpu().double()
    assert (got[:, N:] == 77.0).all(), "written past the end"
    got = got[:, :N]
    fa = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :K]
    fb = b.double() * sb.double().t().repeat_interleave(128, 1)[:, :K].repeat_interleave(
        b_rows, 0)[:N] if b_rows > 1 else b.double() * sb.double().t().repeat_interleave(128, 1)[:, :K]
    x = alpha * (fa @ fb.t()) + (bv.double() if bias else 0)
    size = abs(alpha) * (fa.abs() @ fb.abs().t())
    ref = activation(x, act)
    per = 2.0 ** -11 if fast else 0.0
    err = ((128 + blocks(K) + 16) * U + per) * size + 2 * U * (x.abs() + size)
    if act:
        err = 1.13 * err + 2.0 ** -21 * x.abs()
    fin = torch.finfo(dtype)
    err = err + (ref.abs() + err) * (fin.eps / 2) + fin.smallest_normal * fin.eps
    bad = (got - ref).abs() - err
    assert got.isfinite().all() and bad.max() <= 0, (float(bad.max()), divmod(int(bad.argmax()), N))


SIZES = [(1, 1, 1), (1, 16, 128), (1, 300, 1000), (3, 129, 127), (16, 128, 256), (17, 130, 129),
         (33, 64, 2048), (64, 256, 512), (65, 257, 640), (100, 300, 77), (128, 128, 128),
         (200, 520, 1024), (256, 256, 256), (300, 260, 392), (513, 384, 384), (256, 1024, 2000)]


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, fast):
    check_product(M, N, K, "f32", fast=fast)
    check_product(M, N, K, "bf16", act=lib.ACT_GELU_TANH, fast=fast, pad=-K % 16, seed=2)
    check_product(M, N, K, "f16", act=lib.ACT_SILU, b_rows=1, bias=False, alpha=0.5, fast=fast,
                  seed=3, pad=-K % 16)
    check_product(M, N, K, "f32", b_rows=1, fast=fast, pad=3, offset=5, alpha=-1.5, seed=4)


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("tile", range(11))
@pytest.mark.parametrize("M,N,K", [(256, 256, 256), (512, 384, 1152), (257, 513, 640), (70, 40, 384),
                                   (300, 260, 393), (1, 1, 1), (130, 129, 100), (60, 70, 4240)])
def test_every_tile(M, N, K, tile, fast):
    """Every kernel on whole and ragged tiles, aligned rows and rows off 16-byte boundaries."""
    assert lib.gemm_debug_force_tile(2, tile) == lib.STATUS_SUCCESS
    try:
        check_product(M, N, K, "f32", fast=fast, pad=-K % 16, seed=5)
        check_product(M, N, K, "bf16", act=lib.ACT_GELU_TANH, b_rows=1, fast=fast, pad=-K % 16,
                      seed=6)
        check_product(M, N, K, "f16", fast=fast, pad=1, offset=7, alpha=0.5, bias=False, seed=7)
        check_product(M, N, K, "f32", b_rows=1, fast=fast, pad=3, act=lib.ACT_SILU, seed=8)
    finally:
        lib.gemm_debug_force_tile(2, -1)


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_product_wide_magnitudes(b_rows, fast):
    check_product(130, 140, 1024, "f32", b_rows=b_rows, fast=fast, spread=2.0, seed=9)
    check_product(5, 140, 1024, "f32", b_rows=b_rows, fast=fast, spread=2.0, seed=10)


def test_product_unread_operands():
    C = torch.full((5, 7), 3.0, device="cuda")
    bias = torch.arange(7.0, device="cuda")
    lib.fp8_gemm_bias_act(5, 7, 0, 1.0, None, 1, None, 5, None, 1, None, 1, 128, bias, 0,
                          lib.TYPE_F32, C, 7)
    torch.cuda.synchronize()
    assert torch.equal(C, bias.expand(5, 7))
    lib.fp8_gemm_bias_act(5, 7, 200, 0.0, None, 200, None, 5, None, 200, None, 1, 128, None, 0,
                          lib.TYPE_F32, C, 7, fast_sums=True)
    torch.cuda.synchronize()
    assert (C == 0).all()
    lib.fp8_gemm_bias_act(0, 7, 200, 1.0, None, 200, None, 1, None, 200, None, 1, 128, None, 0,
                          lib.TYPE_F32, None, 7)


@pytest.mark.parametrize("M", [4, 300])
def test_product_propagates_nan_by_element(M):
    N, K = 130, 256
    a, sa, b, sb = operands(M, N, K, 128, 11)
    raw = a.view(torch.uint8)
    raw[2, 100] = 0x7F            # one NaN of A: its row
    sa[1, 3] = float("nan")       # one NaN scale: its row
    C = torch.empty((M, N), device="cuda")
    for fast in (False, True):
        lib.fp8_gemm_bias_act(M, N, K, 1.0, raw.cuda(), K, sa.cuda(), M, b.view(torch.uint8).cuda(),
                              K, sb.cuda(), sb.shape[1], 128, None, 0, lib.TYPE_F32, C, N,
                              fast_sums=fast)
        torch.cuda.synchronize()
        nan = C.cpu().isnan()
        assert nan[2].all() and nan[3].all()
        nan[2:4] = False
        assert not nan.any()


@pytest.mark.parametrize("M,N,K", [(4, 512, 1024), (512, 512, 512)])
def test_quantize_and_product_in_a_graph(M, N, K):
    """Quantise, then multiply, captured once: replays equal the eager calls, bit for bit."""
    x, w = matrix(M, K, "bf16", 1).cuda(), matrix(N, K, "f32", 2).cuda()
    Q, S = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((blocks(K), M),
                                                                              device="cuda")
    W, SW = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty(
        (blocks(K), blocks(N)), device="cuda")
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    lib.fp8_quantize(N, K, lib.TYPE_F32, w, K, 128, W, K, SW, blocks(N))

    def step():
        lib.fp8_quantize(M, K, lib.TYPE_BF16, x, K, 1, Q, K, S, M)
        lib.fp8_gemm_bias_act(M, N, K, 1.0, Q, K, S, M, W, K, SW, blocks(N), 128, None,
                              lib.ACT_SILU, lib.TYPE_BF16, C, N, fast_sums=True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(matrix(M, K, "bf16", 20 + seed))
        step()
        torch.cuda.synchronize()
        want = C.clone()
        C.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)


def test_offsets_past_31_bits():
    """Rows that start more than 2^31 elements into X, A and C."""
    ld = (1 << 30) + 16
    x = torch.randn((3, 128)).to(torch.bfloat16)
    X = torch.zeros((2 * ld + 128,), dtype=torch.bfloat16, device="cuda")
    A = torch.zeros((2 * ld + 128,), dtype=torch.uint8, device="cuda")
    for i in range(3):
        X[i * ld:i * ld + 128] = x[i].cuda()
    S = torch.empty((1, 3), device="cuda")
    lib.fp8_quantize(3, 128, lib.TYPE_BF16, X, ld, 1, A, ld, S, 3)
    q, s = reference(x, 1)
    for i in range(3):
        assert torch.equal(A[i * ld:i * ld + 128].cpu(), q[i].view(torch.uint8))
    lib.fp8_gemm_bias_act(3, 3, 128, 1.0, A, ld, S, 3, A, ld, S, 3, 1, None, 0, lib.TYPE_BF16, X,
                          ld)
    torch.cuda.synchronize()
    f = q.double() * s.double().t()
    want = f @ f.t()
    for i in range(3):
        got = X[i * ld:i * ld + 3].cpu().double()
        assert ((got - want[i]).abs() <= 2.0 ** -8 * want[i].abs() + 200 * U * 128).all()


@pytest.mark.parametrize("M,N,K", [(1000, 3000, 777), (300, 2500, 1024), (2100, 2100, 256)])
def test_tiles_by_the_rule(M, N, K):
    """Enough tiles that the rule leaves the K-split kernels, by every way of summing and scaling."""
    for fast in (False, True):
        for b_rows in (1, 128):
            check_product(M, N, K, "bf16", act=lib.ACT_GELU_TANH, b_rows=b_rows, fast=fast,
                          pad=-K % 16, seed=M + b_rows)
    check_product(M, N, K, "f16", fast=True, pad=1, offset=1, seed=M)


def test_product_on_another_stream():
    M, N, K = 70, 300, 512
    a, sa, b, sb = operands(M, N, K, 128, 21)
    dev = [t.cuda() for t in (a.view(torch.uint8), sa, b.view(torch.uint8), sb)]
    out = [torch.empty((M, N), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for C, stream in zip(out, (None, other)):
        lib.fp8_gemm_bias_act(M, N, K, 1.0, dev[0], K, dev[1], M, dev[2], K, dev[3], 3, 128, None,
                              lib.ACT_SILU, lib.TYPE_F32, C, N, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(*out)
