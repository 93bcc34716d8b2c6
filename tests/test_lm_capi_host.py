"""Refusals of the 8-bit operators and of the mixture-of-experts layer: every bad argument is
answered on the host before the library's state is looked at, so no GPU is needed."""
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


def quantize(**kw):
    a = dict(rows=200, cols=300, type=lib.TYPE_BF16, X=0x1000, ldx=300, block_rows=1, Q=0x2000,
             ldq=300, S=0x3000, lds=200, QT=0x4000, ldqt=200, ST=0x5000, ldst=300)
    a.update(kw)
    return lib.fp8_quantize(stream=0, raise_on_error=False, **a)


def product(**kw):
    a = dict(M=20, N=300, K=130, alpha=1.0, A=0x1000, lda=130, SA=0x2000, ldsa=20, B=0x3000, ldb=130,
             SB=0x4000, ldsb=3, b_rows=128, bias=None, act=0, type=lib.TYPE_F32, C=0x5000, ldc=300)
    a.update(kw)
    return lib.fp8_gemm_bias_act(stream=0, raise_on_error=False, **a)


SHAPE = dict(tokens=3, d_model=100, d_ff=70, experts=8, top_k=2, type=lib.TYPE_BF16,
             weight_type=lib.TYPE_E4M3, act=lib.ACT_SILU, gated=1, norm_topk=0)


def layer(shape=None, **kw):
    a = dict(X=0x1000, ldx=100, R=0x2000, ldr=100, W1=0x3000, ld1=100, S1=0x4000, W2=0x5000, ld2=70,
             S2=0x6000, ids=0x7000, w=0x8000, Y=0x9000, ldy=100, workspace=0x10000,
             workspace_bytes=1 << 20)
    a.update(kw)
    return lib.moe_ffn(lib.MoeShape(**dict(SHAPE, **(shape or {}))), stream=0, raise_on_error=False,
                       **a)


def _id(d):
    return ",".join("%s=%s" % kv for kv in d.items())


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(cols=-1), dict(type=lib.TYPE_E4M3), dict(type=-1), dict(type=7),
    dict(ldx=299), dict(block_rows=0), dict(block_rows=64), dict(block_rows=2), dict(ldq=299),
    dict(lds=199), dict(ldqt=199), dict(ldst=299), dict(X=None), dict(Q=None), dict(S=None),
    dict(QT=None), dict(ST=None), dict(Q=None, S=None, QT=None, ST=None), dict(X=0x1001),
    dict(X=0x1002, type=lib.TYPE_F32), dict(S=0x3002), dict(ST=0x5001),
    dict(block_rows=128, lds=1), dict(block_rows=128, ldst=2),
], ids=_id)
def test_quantize_refuses(bad):
    assert quantize(**bad) == BAD


def test_quantize_accepts():
    assert quantize() == NOT_READY
    assert quantize(Q=None, S=None, ldq=0, lds=0) == NOT_READY
    assert quantize(QT=None, ST=None, ldqt=0, ldst=0) == NOT_READY
    assert quantize(block_rows=128, lds=2, ldst=3) == NOT_READY
    assert quantize(rows=0, X=None) == NOT_READY
    assert quantize(X=0x1002) == NOT_READY


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=129), dict(ldb=129), dict(ldc=299), dict(ldsa=19),
    dict(ldsb=2), dict(b_rows=1, ldsb=299), dict(b_rows=64), dict(b_rows=0), dict(act=3),
    dict(act=-1), dict(type=lib.TYPE_E4M3), dict(type=4), dict(C=None), dict(A=None), dict(B=None),
    dict(SA=None), dict(SB=None), dict(C=0x5002), dict(C=0x5001, type=lib.TYPE_F16),
    dict(SA=0x2001), dict(SB=0x4002), dict(bias=0x6001), dict(fast_sums=2), dict(fast_sums=-1),
], ids=_id)
def test_product_refuses(bad):
    assert product(**bad) == BAD


def test_product_accepts():
    assert product() == NOT_READY
    assert product(b_rows=1, ldsb=300, fast_sums=True, act=lib.ACT_SILU) == NOT_READY
    assert product(A=0x1001, B=0x3003, C=0x5002, type=lib.TYPE_BF16) == NOT_READY
    # alpha == 0 or K == 0: the operands are not read.
    assert product(alpha=0.0, A=None, B=None, SA=None, SB=None) == NOT_READY
    assert product(K=0, A=None, B=None, SA=None, SB=None) == NOT_READY
    assert product(M=0, A=None, B=None, SA=None, SB=None, C=None) == NOT_READY


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=65), dict(d_model=0), dict(d_model=(1 << 20) + 1), dict(d_ff=0),
    dict(d_ff=(1 << 20) + 1), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=9),
    dict(experts=64, top_k=33), dict(type=lib.TYPE_F32, weight_type=lib.TYPE_F32),
    dict(type=lib.TYPE_E4M3), dict(weight_type=lib.TYPE_F16), dict(weight_type=lib.TYPE_F32),
    dict(act=3), dict(act=-1), dict(gated=2), dict(norm_topk=-1),
], ids=_id)
def test_layer_refuses_shapes(bad):
    assert layer(bad) == BAD
    with pytest.raises(lib.GemmError):
        lib.moe_ffn_workspace(lib.MoeShape(**dict(SHAPE, **bad)))


@pytest.mark.parametrize("bad", [
    dict(ldx=99), dict(ldr=99), dict(ld1=99), dict(ld2=69), dict(ldy=99), dict(X=None),
    dict(R=None), dict(W1=None), dict(W2=None), dict(S1=None), dict(S2=None), dict(ids=None),
    dict(w=None), dict(Y=None), dict(workspace=None), dict(workspace_bytes=0), dict(X=0x1001),
    dict(R=0x2001), dict(Y=0x9001), dict(ids=0x7002), dict(w=0x8001), dict(S1=0x4002),
    dict(S2=0x6001), dict(workspace=0x10080),
], ids=_id)
def test_layer_refuses(bad):
    assert layer(**bad) == BAD


def test_layer_accepts():
    assert layer() == NOT_READY
    same = dict(weight_type=lib.TYPE_BF16)
    assert layer(same, S1=None, S2=None) == NOT_READY
    assert layer(same, W1=0x3001) == BAD          # 16-bit weights at an odd address
    assert layer(W1=0x3001) == NOT_READY
    assert layer(dict(tokens=0), X=None, R=None, W1=None, W2=None, ids=None, w=None, Y=None,
                 workspace=None, workspace_bytes=0) == NOT_READY


def test_workspace_size():
    n = lib.moe_ffn_workspace(lib.MoeShape(**SHAPE))
    assert 0 < n < 1 << 20
    assert layer(workspace_bytes=n) == NOT_READY
    assert layer(workspace_bytes=n - 1) == BAD
    assert lib.load_library().moe_ffn_workspace(None, ctypes.byref(ctypes.c_size_t())) == BAD
    assert lib.load_library().moe_ffn_workspace(ctypes.byref(lib.MoeShape(**SHAPE)), None) == BAD


def test_forced_tiles():
    for tile in range(-1, 11):
        assert lib.gemm_debug_force_tile(2, tile) == lib.STATUS_SUCCESS
    assert lib.gemm_debug_force_tile(2, -1) == lib.STATUS_SUCCESS
    assert lib.gemm_debug_force_tile(2, 11) == BAD
    assert lib.gemm_debug_force_tile(2, -2) == BAD
    assert lib.gemm_debug_force_tile(3, 0) == BAD
