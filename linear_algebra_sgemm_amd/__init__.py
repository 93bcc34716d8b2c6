"""Python binding of the MI355X GEMM library (libgemm.so, C ABI in include/gemm.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  Pointers may be given as integers (device
addresses) or as torch tensors (their ``data_ptr()`` is passed; no copy, no
dtype or layout conversion).  ``stream`` may be None (torch's current stream on
the current device), an integer ``hipStream_t`` or a ``torch.cuda.Stream``.

There is no fallback: if libgemm.so has not been built, or the device is not
gfx950, every call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["GemmError", "gemm_create", "gemm_destroy", "sgemm", "sgemm_noalloc", "hgemm_bias_act",
           "bgemm_bias_act", "fp8_quantize", "fp8_gemm_bias_act", "MoeShape", "moe_ffn_workspace",
           "moe_ffn", "i8_quantize", "i8_gemm_bias_act", "i8_gemm_grouped", "moe_sort_workspace",
           "moe_sort", "moe_dispatch", "moe_combine", "moe_combine_grad",
           "gemm_status_string", "gemm_debug_force_tile", "gemm_debug_force_moe_rows",
           "gemm_debug_force_i8_tile",
           "gemm_debug_force_splits",
           "gemm_debug_pick_config", "gemm_debug_use_tuned_table", "gemm_debug_force_swizzle",
           "gemm_debug_tile_map", "library_path",
           "load_library", "EXPORTED_SYMBOLS", "ACT_NONE", "ACT_GELU_TANH", "ACT_SILU",
           "TYPE_F32", "TYPE_F16", "TYPE_BF16", "TYPE_E4M3"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libgemm.so")

STATUS_SUCCESS = 0
STATUS_NOT_INITIALIZED = 1
STATUS_INVALID_VALUE = 2
STATUS_ARCH_MISMATCH = 3
STATUS_HIP_ERROR = 4
STATUS_INTERNAL = 5

ACT_NONE = 0
ACT_GELU_TANH = 1
ACT_SILU = 2   # the 8-bit products and moe_ffn only

TYPE_F32 = 0
TYPE_F16 = 1
TYPE_BF16 = 2
TYPE_E4M3 = 3

# Every symbol declared in include/gemm.h and include/gemm_debug.h.
EXPORTED_SYMBOLS = ("gemm_create", "gemm_destroy", "sgemm", "sgemm_noalloc", "hgemm_bias_act",
                    "bgemm_bias_act", "fp8_quantize", "fp8_gemm_bias_act", "moe_ffn_workspace",
                    "moe_ffn", "i8_quantize", "i8_gemm_bias_act", "i8_gemm_grouped",
                    "moe_sort_workspace", "moe_sort", "moe_dispatch", "moe_combine",
                    "moe_combine_grad",
                    "gemm_status_string", "gemm_debug_force_tile", "gemm_debug_force_moe_rows",
                    "gemm_debug_force_i8_tile",
                    "gemm_debug_force_splits",
                    "gemm_debug_pick_config", "gemm_debug_use_tuned_table",
                    "gemm_debug_force_swizzle", "gemm_debug_tile_map")

_lib = None


class MoeShape(ctypes.Structure):
    """moe_shape_t of include/gemm.h; every field by keyword."""
    _fields_ = [(n, ctypes.c_int) for n in ("tokens", "d_model", "d_ff", "experts", "top_k", "type",
                                            "weight_type", "act", "gated", "norm_topk")]


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: status %d (%s)" % (where, status, gemm_status_string(status)))


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libgemm.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libgemm.so is not built (run `python -m linear_algebra_sgemm_amd.build` "
                           "or __graft_entry__.build()); there is no non-HIP fallback")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.gemm_create.argtypes = []
    lib.gemm_create.restype = I
    lib.gemm_destroy.argtypes = []
    lib.gemm_destroy.restype = I
    lib.sgemm.argtypes = [I, I, I, F, P, I, P, I, F, P, I, P]
    lib.sgemm.restype = I
    lib.sgemm_noalloc.argtypes = [I, I, I, F, P, I, P, I, F, P, I, P]
    lib.sgemm_noalloc.restype = I
    lib.hgemm_bias_act.argtypes = [I, I, I, F, P, I, P, I, P, I, P, I, P]
    lib.hgemm_bias_act.restype = I
    lib.bgemm_bias_act.argtypes = [I, I, I, F, P, I, P, I, P, I, P, I, P]
    lib.bgemm_bias_act.restype = I
    S, SP = ctypes.c_size_t, ctypes.POINTER(MoeShape)
    lib.fp8_quantize.argtypes = [I, I, I, P, I, I, P, I, P, I, P, I, P, I, P]
    lib.fp8_quantize.restype = I
    lib.fp8_gemm_bias_act.argtypes = [I, I, I, F, P, I, P, I, P, I, P, I, I, P, I, I, P, I, I, P]
    lib.fp8_gemm_bias_act.restype = I
    lib.moe_ffn_workspace.argtypes = [SP, ctypes.POINTER(S)]
    lib.moe_ffn_workspace.restype = I
    lib.moe_ffn.argtypes = [SP, P, I, P, I, P, I, P, P, I, P, P, P, P, I, P, S, P]
    lib.moe_ffn.restype = I
    lib.i8_quantize.argtypes = [I, I, I, P, I, P, I, P, P]
    lib.i8_quantize.restype = I
    lib.i8_gemm_bias_act.argtypes = [I, I, I, F, P, I, P, P, I, P, P, I, I, I, P, I, P]
    lib.i8_gemm_bias_act.restype = I
    lib.i8_gemm_grouped.argtypes = [I, P, I, I, I, F, P, I, P, I, P, I, P, I, P, P, I, I, I, P, I, P]
    lib.i8_gemm_grouped.restype = I
    lib.moe_sort_workspace.argtypes = [I, I, I, ctypes.POINTER(S)]
    lib.moe_sort_workspace.restype = I
    lib.moe_sort.argtypes = [I, I, I, P, P, P, P, P, S, P]
    lib.moe_sort.restype = I
    lib.moe_dispatch.argtypes = [I, I, I, I, P, I, P, P, P, I, I, P]
    lib.moe_dispatch.restype = I
    lib.moe_combine.argtypes = [I, I, I, I, P, I, I, P, P, P, I, P]
    lib.moe_combine.restype = I
    lib.moe_combine_grad.argtypes = [I, I, I, I, P, I, P, I, I, P, P, P, I, P, P]
    lib.moe_combine_grad.restype = I
    lib.gemm_debug_force_i8_tile.argtypes = [I]
    lib.gemm_debug_force_i8_tile.restype = I
    lib.gemm_status_string.argtypes = [I]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_debug_force_tile.argtypes = [I, I]
    lib.gemm_debug_force_tile.restype = I
    lib.gemm_debug_force_moe_rows.argtypes = [I]
    lib.gemm_debug_force_moe_rows.restype = I
    lib.gemm_debug_force_splits.argtypes = [I, I]
    lib.gemm_debug_force_splits.restype = I
    IP = ctypes.POINTER(ctypes.c_int)
    lib.gemm_debug_pick_config.argtypes = [I, I, I, I, I, IP, IP]
    lib.gemm_debug_pick_config.restype = I
    lib.gemm_debug_use_tuned_table.argtypes = [I]
    lib.gemm_debug_use_tuned_table.restype = I
    lib.gemm_debug_force_swizzle.argtypes = [I, I]
    lib.gemm_debug_force_swizzle.restype = I
    lib.gemm_debug_tile_map.argtypes = [I, I, I, I, P, P]
    lib.gemm_debug_tile_map.restype = I
    _lib = lib
    return lib


def _ptr(x):
    if x is None or type(x) is int:
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, int):
        return int(x)
    raise TypeError("expected a device pointer (int) or a tensor, got %r" % type(x))


_raw_stream = None   # torch's current stream on the current device, as an integer


def _find_raw_stream():
    """torch.cuda.current_stream() builds a Stream object, about 2 us of every call; where torch
    offers the bare handle (as its own compiled code uses it), that is taken instead."""
    global _raw_stream
    import torch
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if stream is not None and device is not None and torch.cuda.is_initialized():
        _raw_stream = lambda: stream(device())   # noqa: E731
        return _raw_stream()
    return torch.cuda.current_stream().cuda_stream


def _stream(stream):
    if stream is None:
        return _find_raw_stream() if _raw_stream is None else _raw_stream()
    if isinstance(stream, int):
        return stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    raise TypeError("expected None, an int hipStream_t or a torch.cuda.Stream")


def _check(status: int, where: str, raise_on_error: bool) -> int:
    if status != STATUS_SUCCESS and raise_on_error:
        raise GemmError(status, where)
    return status


def gemm_create(raise_on_error: bool = True) -> int:
    return _check(load_library().gemm_create(), "gemm_create", raise_on_error)


def gemm_destroy(raise_on_error: bool = True) -> int:
    return _check(load_library().gemm_destroy(), "gemm_destroy", raise_on_error)


def sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None, *, raise_on_error=True):
    """C = alpha * A x B + beta * C (FP32, row-major); see include/gemm.h."""
    st = load_library().sgemm(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda), _ptr(B),
                              int(ldb), float(beta), _ptr(C), int(ldc), _stream(stream))
    return _check(st, "sgemm", raise_on_error)


def sgemm_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None, *,
                  raise_on_error=True):
    """sgemm without device allocation on the call path; see include/gemm.h."""
    st = load_library().sgemm_noalloc(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                      _ptr(B), int(ldb), float(beta), _ptr(C), int(ldc),
                                      _stream(stream))
    return _check(st, "sgemm_noalloc", raise_on_error)


def hgemm_bias_act(M, N, K, alpha, A, lda, B, ldb, bias, act, C, ldc, stream=None, *,
                   raise_on_error=True):
    """C = act(alpha * A x B + bias), fp16 A/B/C, fp32 bias and accumulation; see include/gemm.h."""
    st = load_library().hgemm_bias_act(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                       _ptr(B), int(ldb), _ptr(bias), int(act), _ptr(C), int(ldc),
                                       _stream(stream))
    return _check(st, "hgemm_bias_act", raise_on_error)


def bgemm_bias_act(M, N, K, alpha, A, lda, B, ldb, bias, act, C, ldc, stream=None, *,
                   raise_on_error=True):
    """C = act(alpha * A x B + bias), bfloat16 A/B/C, fp32 bias and accumulation; see include/gemm.h."""
    st = load_library().bgemm_bias_act(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                       _ptr(B), int(ldb), _ptr(bias), int(act), _ptr(C), int(ldc),
                                       _stream(stream))
    return _check(st, "bgemm_bias_act", raise_on_error)


def fp8_quantize(rows, cols, type, X, ldx, block_rows, Q, ldq, S, lds, QT=None, ldqt=0, ST=None,
                 ldst=0, stream=None, *, raise_on_error=True):
    """e4m3 values and block scales of X and / or of its transpose; see include/gemm.h."""
    st = load_library().fp8_quantize(int(rows), int(cols), int(type), _ptr(X), int(ldx),
                                     int(block_rows), _ptr(Q), int(ldq), _ptr(S), int(lds),
                                     _ptr(QT), int(ldqt), _ptr(ST), int(ldst), _stream(stream))
    return _check(st, "fp8_quantize", raise_on_error)


def fp8_gemm_bias_act(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, b_rows, bias, act, type, C,
                      ldc, stream=None, *, fast_sums=False, raise_on_error=True):
    """C = act(alpha * A x B^T + bias), block-scaled e4m3 A and B; see include/gemm.h.

    fast_sums: let the 8-bit matrix instructions form each block's sum (twice the rate; each product
    to 13 bits below the largest of eight columns, at worst 8.6e-4 of sum |a||b|): for 16-bit results."""
    st = load_library().fp8_gemm_bias_act(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                          _ptr(SA), int(ldsa), _ptr(B), int(ldb), _ptr(SB),
                                          int(ldsb), int(b_rows), _ptr(bias), int(act), int(type),
                                          _ptr(C), int(ldc), int(fast_sums), _stream(stream))
    return _check(st, "fp8_gemm_bias_act", raise_on_error)


def moe_ffn_workspace(shape: MoeShape) -> int:
    """Bytes of device memory a moe_ffn call of this shape needs as its workspace."""
    n = ctypes.c_size_t(0)
    _check(load_library().moe_ffn_workspace(ctypes.byref(shape), ctypes.byref(n)),
           "moe_ffn_workspace", True)
    return n.value


def moe_ffn(shape, X, ldx, R, ldr, W1, ld1, S1, W2, ld2, S2, ids, w, Y, ldy, workspace,
            workspace_bytes, stream=None, *, raise_on_error=True):
    """A mixture-of-experts feed-forward layer for up to 64 tokens; see include/gemm.h."""
    st = load_library().moe_ffn(ctypes.byref(shape), _ptr(X), int(ldx), _ptr(R), int(ldr), _ptr(W1),
                                int(ld1), _ptr(S1), _ptr(W2), int(ld2), _ptr(S2), _ptr(ids),
                                _ptr(w), _ptr(Y), int(ldy), _ptr(workspace), int(workspace_bytes),
                                _stream(stream))
    return _check(st, "moe_ffn", raise_on_error)


def i8_quantize(rows, cols, type, X, ldx, Q, ldq, S, stream=None, *, raise_on_error=True):
    """Rows of X as int8 values and a scale for each row; see include/gemm.h."""
    st = load_library().i8_quantize(int(rows), int(cols), int(type), _ptr(X), int(ldx), _ptr(Q),
                                    int(ldq), _ptr(S), _stream(stream))
    return _check(st, "i8_quantize", raise_on_error)


def i8_gemm_bias_act(M, N, K, alpha, A, lda, SA, B, ldb, SB, bias, act, gated, type, C, ldc,
                     stream=None, *, raise_on_error=True):
    """C = act(alpha SA SB A x B^T + bias), int8 A and B with a scale for every row; gated: times the
    product's second N columns; see include/gemm.h."""
    st = load_library().i8_gemm_bias_act(int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                         _ptr(SA), _ptr(B), int(ldb), _ptr(SB), _ptr(bias), int(act),
                                         int(gated), int(type), _ptr(C), int(ldc), _stream(stream))
    return _check(st, "i8_gemm_bias_act", raise_on_error)


def i8_gemm_grouped(groups, offsets, M, N, K, alpha, A, lda, SA, a_rows, index, per, B, ldb, SB, bias,
                    act, gated, type, C, ldc, stream=None, *, raise_on_error=True):
    """i8_gemm_bias_act of rows in groups, each with a matrix of its own; see include/gemm.h."""
    st = load_library().i8_gemm_grouped(int(groups), _ptr(offsets), int(M), int(N), int(K),
                                        float(alpha), _ptr(A), int(lda), _ptr(SA), int(a_rows),
                                        _ptr(index), int(per), _ptr(B), int(ldb), _ptr(SB),
                                        _ptr(bias), int(act), int(gated), int(type), _ptr(C),
                                        int(ldc), _stream(stream))
    return _check(st, "i8_gemm_grouped", raise_on_error)


def moe_sort_workspace(tokens, top_k, experts) -> int:
    """Bytes of device memory a moe_sort call of this shape needs as its workspace."""
    n = ctypes.c_size_t(0)
    _check(load_library().moe_sort_workspace(int(tokens), int(top_k), int(experts), ctypes.byref(n)),
           "moe_sort_workspace", True)
    return n.value


def moe_sort(tokens, top_k, experts, ids, offsets, src, pos, workspace, workspace_bytes, stream=None,
             *, raise_on_error=True):
    """Entries (token, slot) in the order of their experts; see include/gemm.h."""
    st = load_library().moe_sort(int(tokens), int(top_k), int(experts), _ptr(ids), _ptr(offsets),
                                 _ptr(src), _ptr(pos), _ptr(workspace), int(workspace_bytes),
                                 _stream(stream))
    return _check(st, "moe_sort", raise_on_error)


def moe_dispatch(tokens, top_k, cols, type, X, ldx, pos, w, Y, ldy, y_rows, stream=None, *,
                 raise_on_error=True):
    """Y[pos[t][s]] = X[t], times w[t][s] if given; see include/gemm.h."""
    st = load_library().moe_dispatch(int(tokens), int(top_k), int(cols), int(type), _ptr(X), int(ldx),
                                     _ptr(pos), _ptr(w), _ptr(Y), int(ldy), int(y_rows),
                                     _stream(stream))
    return _check(st, "moe_dispatch", raise_on_error)


def moe_combine(tokens, top_k, cols, type, X, ldx, x_rows, pos, w, Y, ldy, stream=None, *,
                raise_on_error=True):
    """Y[t] = sum_s w[t][s] X[pos[t][s]]; see include/gemm.h."""
    st = load_library().moe_combine(int(tokens), int(top_k), int(cols), int(type), _ptr(X), int(ldx),
                                    int(x_rows), _ptr(pos), _ptr(w), _ptr(Y), int(ldy),
                                    _stream(stream))
    return _check(st, "moe_combine", raise_on_error)


def moe_combine_grad(tokens, top_k, cols, type, dY, lddy, X, ldx, x_rows, pos, w, dX, lddx, dw,
                     stream=None, *, raise_on_error=True):
    """moe_combine's gradients to its rows and its weights; see include/gemm.h."""
    st = load_library().moe_combine_grad(int(tokens), int(top_k), int(cols), int(type), _ptr(dY),
                                         int(lddy), _ptr(X), int(ldx), int(x_rows), _ptr(pos),
                                         _ptr(w), _ptr(dX), int(lddx), _ptr(dw), _stream(stream))
    return _check(st, "moe_combine_grad", raise_on_error)


def gemm_status_string(status: int) -> str:
    try:
        return load_library().gemm_status_string(int(status)).decode()
    except RuntimeError:
        return "status %d" % status


def gemm_debug_force_tile(op: int, tile: int) -> int:
    return load_library().gemm_debug_force_tile(int(op), int(tile))


def gemm_debug_force_moe_rows(rows: int) -> int:
    return load_library().gemm_debug_force_moe_rows(int(rows))


def gemm_debug_force_i8_tile(tile: int) -> int:
    return load_library().gemm_debug_force_i8_tile(int(tile))


def gemm_debug_force_splits(op: int, splits: int) -> int:
    return load_library().gemm_debug_force_splits(int(op), int(splits))


def gemm_debug_use_tuned_table(on: bool) -> int:
    return load_library().gemm_debug_use_tuned_table(1 if on else 0)


def gemm_debug_pick_config(op: int, M: int, N: int, K: int, cus: int):
    """(tile, splits) the library would run for this shape, or raise GemmError."""
    tile, splits = ctypes.c_int(-1), ctypes.c_int(-1)
    st = load_library().gemm_debug_pick_config(int(op), int(M), int(N), int(K), int(cus),
                                                ctypes.byref(tile), ctypes.byref(splits))
    _check(st, "gemm_debug_pick_config", True)
    return tile.value, splits.value


def gemm_debug_force_swizzle(group_m: int, xcd_remap: bool = True) -> int:
    """Tile order of later launches: group_m 0 = each launch's own; see include/gemm_debug.h."""
    return load_library().gemm_debug_force_swizzle(int(group_m), 1 if xcd_remap else 0)


def gemm_debug_tile_map(tiles_m: int, tiles_n: int, group_m: int, xcd_remap: bool = True):
    """(tile_m, tile_n) int arrays: the output tile of every workgroup of such a launch."""
    import numpy as np
    n = int(tiles_m) * int(tiles_n)
    tm = np.empty(max(n, 1), np.int32)
    tn = np.empty(max(n, 1), np.int32)
    st = load_library().gemm_debug_tile_map(int(tiles_m), int(tiles_n), int(group_m),
                                            1 if xcd_remap else 0, tm.ctypes.data, tn.ctypes.data)
    _check(st, "gemm_debug_tile_map", True)
    return tm[:n], tn[:n]
