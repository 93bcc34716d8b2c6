"""Refusals of the int8 operators and of the exchange of tokens with the experts' order: every bad
argument is answered on the host before the library's state is looked at, so no GPU is needed."""
import ctypes
import os

import pytest

import linear_algebra_sgemm_amd as lib

BAD, NOT_READY = lib.STATUS_INVALID_VALUE, lib.STATUS_NOT_INITIALIZED


@pytest.fixture(scope="module", autouse=True)
def so():
    if not os.path.exists(lib.library_path()):
        pytest.fail("libgemm.so is not built; run __graft_entry__.build() first")
    return lib.load_library()


def caller(fn, **defaults):
    def call(**kw):
        return fn(stream=0, raise_on_error=False, **dict(defaults, **kw))
    return call


quantize = caller(lib.i8_quantize, rows=200, cols=300, type=lib.TYPE_BF16, X=0x1000, ldx=300, Q=0x2000,
                  ldq=300, S=0x3000)
product = caller(lib.i8_gemm_bias_act, M=20, N=300, K=130, alpha=1.0, A=0x1000, lda=130, SA=0x2000,
                 B=0x3000, ldb=130, SB=0x4000, bias=None, act=0, gated=0, type=lib.TYPE_F32, C=0x5000,
                 ldc=300)
grouped = caller(lib.i8_gemm_grouped, groups=8, offsets=0x8000, M=20, N=300, K=130, alpha=1.0, A=0x1000,
                 lda=130, SA=0x2000, a_rows=20, index=None, per=1, B=0x3000, ldb=130, SB=0x4000,
                 bias=None, act=0, gated=0, type=lib.TYPE_F32, C=0x5000, ldc=300)
sort = caller(lib.moe_sort, tokens=100, top_k=4, experts=8, ids=0x1000, offsets=0x2000, src=0x3000,
              pos=0x4000, workspace=0x10000, workspace_bytes=1 << 24)
dispatch = caller(lib.moe_dispatch, tokens=10, top_k=4, cols=100, type=lib.TYPE_BF16, X=0x1000, ldx=100,
                  pos=0x2000, w=0x3000, Y=0x4000, ldy=100, y_rows=40)
combine = caller(lib.moe_combine, tokens=10, top_k=4, cols=100, type=lib.TYPE_BF16, X=0x1000, ldx=100,
                 x_rows=40, pos=0x2000, w=0x3000, Y=0x4000, ldy=100)
grad = caller(lib.moe_combine_grad, tokens=10, top_k=4, cols=100, type=lib.TYPE_BF16, dY=0x1000, lddy=100,
              X=0x2000, ldx=100, x_rows=40, pos=0x3000, w=0x4000, dX=0x5000, lddx=100, dw=0x6000)


def _id(d):
    return ",".join("%s=%s" % kv for kv in d.items())


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(cols=-1), dict(cols=(1 << 20) + 1, ldx=1 << 21, ldq=1 << 21),
    dict(type=lib.TYPE_E4M3), dict(type=-1), dict(type=4), dict(ldx=299), dict(ldq=299), dict(X=None),
    dict(Q=None), dict(S=None), dict(X=0x1001), dict(X=0x1002, type=lib.TYPE_F32), dict(S=0x3002),
    dict(cols=0, ldx=0), dict(cols=0, ldq=0),
], ids=_id)
def test_quantize_refuses(bad):
    assert quantize(**bad) == BAD


def test_quantize_accepts():
    assert quantize() == NOT_READY
    assert quantize(Q=0x2001, X=0x1002) == NOT_READY
    assert quantize(rows=0, X=None, Q=None, S=None) == NOT_READY
    assert quantize(cols=1 << 20, ldx=1 << 20, ldq=1 << 20) == NOT_READY


COMMON = [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(K=131072, lda=131072, ldb=131072), dict(lda=129),
    dict(ldb=129), dict(ldc=299), dict(act=3), dict(act=-1), dict(gated=2), dict(gated=-1),
    dict(type=lib.TYPE_E4M3), dict(type=-1), dict(type=4), dict(C=None), dict(A=None), dict(B=None),
    dict(SA=None), dict(SB=None), dict(C=0x5002), dict(C=0x5001, type=lib.TYPE_F16), dict(SA=0x2001),
    dict(SB=0x4002), dict(bias=0x6001), dict(gated=1, N=(1 << 30) + 1, ldc=(1 << 30) + 1),
]


@pytest.mark.parametrize("bad", COMMON, ids=_id)
def test_products_refuse(bad):
    assert product(**bad) == BAD
    assert grouped(**bad) == BAD


@pytest.mark.parametrize("bad", [
    dict(groups=-1), dict(groups=1025), dict(offsets=None), dict(offsets=0x8002), dict(per=0),
    dict(per=-1), dict(a_rows=19), dict(a_rows=-1, index=0x9000), dict(a_rows=0, index=0x9000),
    dict(index=0x9001),
], ids=_id)
def test_grouped_refuses(bad):
    assert grouped(**bad) == BAD


def test_products_accept():
    for call in (product, grouped):
        assert call() == NOT_READY
        assert call(gated=1, act=lib.ACT_SILU, bias=0x6000) == NOT_READY
        assert call(A=0x1001, B=0x3003, C=0x5002, type=lib.TYPE_BF16) == NOT_READY
        assert call(K=131071, lda=131071, ldb=131071) == NOT_READY
        # alpha == 0 or K == 0: the operands are not read.
        assert call(alpha=0.0, A=None, B=None, SA=None, SB=None) == NOT_READY
        assert call(K=0, A=None, B=None, SA=None, SB=None) == NOT_READY
        assert call(M=0, A=None, B=None, SA=None, SB=None, C=None) == NOT_READY
        assert call(N=0, ldc=1, A=None, B=None, SA=None, SB=None, C=None) == NOT_READY
    assert grouped(index=0x9000, per=8, a_rows=3) == NOT_READY
    assert grouped(groups=0, offsets=None, C=None, A=None, B=None, SA=None, SB=None) == NOT_READY
    assert grouped(groups=1024) == NOT_READY


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(top_k=0), dict(top_k=33), dict(experts=0), dict(experts=1025),
    dict(tokens=(1 << 30) // 4 + 1), dict(tokens=(1 << 31) - 1), dict(ids=None), dict(offsets=None),
    dict(src=None), dict(pos=None), dict(workspace=None), dict(workspace_bytes=0), dict(ids=0x1002),
    dict(offsets=0x2001), dict(src=0x3002), dict(pos=0x4001), dict(workspace=0x10080),
], ids=_id)
def test_sort_refuses(bad):
    assert sort(**bad) == BAD


def test_sort_accepts():
    assert sort() == NOT_READY
    assert sort(experts=2, top_k=32) == NOT_READY
    assert sort(tokens=0, ids=None, src=None, pos=None, workspace=None, workspace_bytes=0) == NOT_READY
    assert sort(tokens=0, offsets=None) == BAD


def test_sort_workspace():
    for shape in ((0, 1, 1), (1, 8, 64), (300, 4, 8), (5000, 32, 1024)):
        n = lib.moe_sort_workspace(*shape)
        assert 0 < n <= 1 << 21
        args = dict(zip(("tokens", "top_k", "experts"), shape))
        assert sort(workspace_bytes=n, **args) == NOT_READY
        if shape[0]:
            assert sort(workspace_bytes=n - 1, **args) == BAD
    for shape in ((-1, 1, 1), (1, 0, 1), (1, 33, 1), (1, 1, 0), (1, 1, 1025), (1 << 29, 4, 8)):
        with pytest.raises(lib.GemmError):
            lib.moe_sort_workspace(*shape)
    assert lib.load_library().moe_sort_workspace(1, 1, 1, None) == BAD


EXCHANGE = [dict(tokens=-1), dict(top_k=0), dict(top_k=33), dict(cols=-1), dict(type=lib.TYPE_E4M3),
            dict(type=4), dict(type=-1), dict(pos=None), dict(pos=0x2002), dict(w=0x3002), dict(X=None),
            dict(X=0x1001), dict(X=0x1002, type=lib.TYPE_F32), dict(ldx=99)]


@pytest.mark.parametrize("bad", EXCHANGE + [dict(y_rows=-1), dict(Y=None), dict(Y=0x4001), dict(ldy=99)],
                         ids=_id)
def test_dispatch_refuses(bad):
    assert dispatch(**bad) == BAD


@pytest.mark.parametrize("bad", EXCHANGE + [dict(x_rows=-1), dict(Y=None), dict(Y=0x4001), dict(ldy=99)],
                         ids=_id)
def test_combine_refuses(bad):
    assert combine(**bad) == BAD


@pytest.mark.parametrize("bad", EXCHANGE + [
    dict(x_rows=-1), dict(dY=None), dict(dY=0x1001), dict(lddy=99), dict(dX=0x5001), dict(lddx=99),
    dict(dw=0x6002), dict(dX=None, dw=None)], ids=_id)
def test_grad_refuses(bad):
    assert grad(**bad) == BAD


def test_exchange_accepts():
    for call in (dispatch, combine, grad):
        assert call() == NOT_READY
        assert call(w=None) == NOT_READY
        assert call(tokens=0) == NOT_READY
    assert dispatch(y_rows=0, X=None, Y=None) == NOT_READY
    assert dispatch(cols=0, X=None, Y=None, pos=None) == NOT_READY
    assert combine(x_rows=0, X=None) == NOT_READY
    assert combine(tokens=0, X=None, pos=None, Y=None) == NOT_READY
    assert grad(dX=None, lddx=0) == NOT_READY
    assert grad(dw=None, X=None, ldx=0) == NOT_READY
    assert grad(x_rows=0, X=None, dY=None, dX=None) == NOT_READY
    assert grad(tokens=0, dY=None, X=None, pos=None, w=None, dX=None, dw=None) == NOT_READY


def test_forced_tiles():
    for tile in range(-1, 12):
        assert lib.gemm_debug_force_i8_tile(tile) == lib.STATUS_SUCCESS
    assert lib.gemm_debug_force_i8_tile(-1) == lib.STATUS_SUCCESS
    assert lib.gemm_debug_force_i8_tile(12) == BAD
    assert lib.gemm_debug_force_i8_tile(-2) == BAD


def test_null_shape_pointer():
    assert lib.load_library().moe_sort_workspace(4, 2, 8, ctypes.byref(ctypes.c_size_t())) == 0
