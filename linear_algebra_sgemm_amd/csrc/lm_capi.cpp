// C ABI of the 8-bit operators, the mixture-of-experts layer and the exchange of
// tokens with the experts' order (declared in include/gemm.h): argument checks,
// quick returns, and the launch.  None of these calls allocates, copies to the host or
// uses the library's own workspace, so all may be captured into a graph and run on any stream.
#include <atomic>
#include <cmath>

#include "../../include/gemm_debug.h"
#include "lm_launch.h"

namespace {

std::atomic<int> g_force_moe_rows{0};
std::atomic<int> g_force_i8_tile{-1};

constexpr int kMaxI8K = 131071;         // 2^14 K stays below 2^31
constexpr int kMaxI8Cols = 1 << 20;     // of a row that i8_quantize takes
constexpr int kMaxExperts = 1024, kMaxTopK = 32;
constexpr int64_t kMaxEntries = 1 << 30;   // of a sort

bool ld_ok(int ld, int cols) { return ld >= (cols > 1 ? cols : 1); }
int blocks(int n) { return (int)(((int64_t)n + 127) / 128); }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool flag_ok(int x) { return x == 0 || x == 1; }
bool act_ok(int act) {
  return act == GEMM_ACT_NONE || act == GEMM_ACT_GELU_TANH || act == GEMM_ACT_SILU;
}
bool float_type(int t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_F16 || t == GEMM_TYPE_BF16; }
uintptr_t elem(int type) { return type == GEMM_TYPE_F32 ? 4 : type == GEMM_TYPE_E4M3 ? 1 : 2; }

int finish(hipError_t e) {
  return e == hipSuccess ? GEMM_STATUS_SUCCESS : lasg::library_hip_failure(e);
}

bool shape_ok(const moe_shape_t& s) {
  return s.tokens >= 0 && s.tokens <= 64 && s.d_model >= 1 && s.d_model <= (1 << 20) &&
         s.d_ff >= 1 && s.d_ff <= (1 << 20) && s.experts >= 1 && s.experts <= 1024 &&
         s.top_k >= 1 && s.top_k <= 32 && s.top_k <= s.experts &&
         (s.type == GEMM_TYPE_F16 || s.type == GEMM_TYPE_BF16) &&
         (s.weight_type == s.type || s.weight_type == GEMM_TYPE_E4M3) && act_ok(s.act) &&
         flag_ok(s.gated) && flag_ok(s.norm_topk);
}

}  // namespace

extern "C" {

int fp8_quantize(int rows, int cols, int type, const void* X, int ldx, int block_rows, uint8_t* Q,
                 int ldq, float* S, int lds, uint8_t* QT, int ldqt, float* ST, int ldst,
                 hipStream_t stream) {
  if (rows < 0 || cols < 0 || !float_type(type) || !ld_ok(ldx, cols))
    return GEMM_STATUS_INVALID_VALUE;
  if (block_rows != 1 && block_rows != 128) return GEMM_STATUS_INVALID_VALUE;
  const bool empty = rows == 0 || cols == 0;
  // (An empty array may well have a null pointer.)
  if (!empty && ((Q == nullptr) != (S == nullptr) || (QT == nullptr) != (ST == nullptr)))
    return GEMM_STATUS_INVALID_VALUE;
  if (!empty && (X == nullptr || (Q == nullptr && QT == nullptr))) return GEMM_STATUS_INVALID_VALUE;
  if (Q != nullptr && (!ld_ok(ldq, cols) || !ld_ok(lds, block_rows == 1 ? rows : blocks(rows))))
    return GEMM_STATUS_INVALID_VALUE;
  if (QT != nullptr && (!ld_ok(ldqt, rows) || !ld_ok(ldst, block_rows == 1 ? cols : blocks(cols))))
    return GEMM_STATUS_INVALID_VALUE;
  if (!aligned(X, elem(type)) || !aligned(S, 4) || !aligned(ST, 4))
    return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (empty) return GEMM_STATUS_SUCCESS;
  const lasg::QuantizeCall c{rows, cols, type, X, ldx, block_rows, Q, ldq, S, lds, QT, ldqt, ST,
                             ldst};
  return finish(lasg::launch_quantize(c, stream));
}

int fp8_gemm_bias_act(int M, int N, int K, float alpha, const uint8_t* A, int lda, const float* SA,
                      int ldsa, const uint8_t* B, int ldb, const float* SB, int ldsb, int b_rows,
                      const float* bias, int act, int type, void* C, int ldc, int fast_sums,
                      hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return GEMM_STATUS_INVALID_VALUE;
  if (!ld_ok(lda, K) || !ld_ok(ldb, K) || !ld_ok(ldc, N)) return GEMM_STATUS_INVALID_VALUE;
  if (b_rows != 1 && b_rows != 128) return GEMM_STATUS_INVALID_VALUE;
  if (!ld_ok(ldsa, M) || !ld_ok(ldsb, b_rows == 1 ? N : blocks(N)))
    return GEMM_STATUS_INVALID_VALUE;
  if (!act_ok(act) || !float_type(type) || !flag_ok(fast_sums)) return GEMM_STATUS_INVALID_VALUE;
  const bool empty = M == 0 || N == 0;
  const bool reads_ab = !empty && K > 0 && alpha != 0.0f;
  if (!empty && C == nullptr) return GEMM_STATUS_INVALID_VALUE;
  if (reads_ab && (A == nullptr || B == nullptr || SA == nullptr || SB == nullptr))
    return GEMM_STATUS_INVALID_VALUE;
  if (!aligned(C, elem(type)) || !aligned(SA, 4) || !aligned(SB, 4) || !aligned(bias, 4))
    return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (empty) return GEMM_STATUS_SUCCESS;
  const lasg::Fp8Call c{M, N, reads_ab ? K : 0, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, b_rows,
                        bias, act, type, C, ldc, fast_sums == 1};
  return finish(
      lasg::launch_fp8_gemm(c, lasg::library_cus(), lasg::library_force_fp8_tile(), stream));
}

int moe_ffn_workspace(const moe_shape_t* shape, size_t* bytes) {
  if (shape == nullptr || bytes == nullptr || !shape_ok(*shape)) return GEMM_STATUS_INVALID_VALUE;
  *bytes = lasg::moe_workspace_bytes(*shape);
  return GEMM_STATUS_SUCCESS;
}

int moe_ffn(const moe_shape_t* shape, const uint16_t* X, int ldx, const uint16_t* R, int ldr,
            const void* W1, int ld1, const float* S1, const void* W2, int ld2, const float* S2,
            int* ids, float* w, uint16_t* Y, int ldy, void* workspace, size_t workspace_bytes,
            hipStream_t stream) {
  if (shape == nullptr || !shape_ok(*shape)) return GEMM_STATUS_INVALID_VALUE;
  const moe_shape_t& s = *shape;
  if (ldx < s.d_model || ldr < s.d_model || ld1 < s.d_model || ld2 < s.d_ff || ldy < s.d_model)
    return GEMM_STATUS_INVALID_VALUE;
  const bool fp8 = s.weight_type == GEMM_TYPE_E4M3;
  if (s.tokens > 0) {
    if (X == nullptr || R == nullptr || W1 == nullptr || W2 == nullptr || ids == nullptr ||
        w == nullptr || Y == nullptr || workspace == nullptr)
      return GEMM_STATUS_INVALID_VALUE;
    if (fp8 && (S1 == nullptr || S2 == nullptr)) return GEMM_STATUS_INVALID_VALUE;
    if (workspace_bytes < lasg::moe_workspace_bytes(s)) return GEMM_STATUS_INVALID_VALUE;
  }
  if (!aligned(X, 2) || !aligned(R, 2) || !aligned(Y, 2) || !aligned(W1, elem(s.weight_type)) ||
      !aligned(W2, elem(s.weight_type)) || !aligned(ids, 4) || !aligned(w, 4) ||
      (fp8 && (!aligned(S1, 4) || !aligned(S2, 4))) || !aligned(workspace, 256))
    return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (s.tokens == 0) return GEMM_STATUS_SUCCESS;
  const lasg::MoeCall c{s, X, ldx, R, ldr, W1, ld1, S1, W2, ld2, S2, ids, w, Y, ldy, workspace};
  return finish(lasg::launch_moe(c, lasg::library_cus(), g_force_moe_rows.load(), stream));
}

int i8_quantize(int rows, int cols, int type, const void* X, int ldx, int8_t* Q, int ldq, float* S,
                hipStream_t stream) {
  if (rows < 0 || cols < 0 || cols > kMaxI8Cols || !float_type(type) || !ld_ok(ldx, cols) ||
      !ld_ok(ldq, cols))
    return GEMM_STATUS_INVALID_VALUE;
  const bool empty = rows == 0 || cols == 0;
  if (!empty && (X == nullptr || Q == nullptr || S == nullptr)) return GEMM_STATUS_INVALID_VALUE;
  if (!aligned(X, elem(type)) || !aligned(S, 4)) return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (empty) return GEMM_STATUS_SUCCESS;
  const lasg::I8QuantizeCall c{rows, cols, type, X, ldx, Q, ldq, S};
  return finish(lasg::launch_i8_quantize(c, lasg::library_cus(), stream));
}

}  // extern "C"

namespace {

// Both forms of the int8 product; groups 0: no groups.
int i8_product(bool grouped, int groups, const int* offsets, int M, int N, int K, float alpha,
               const int8_t* A, int lda, const float* SA, int a_rows, const int* index, int per,
               const int8_t* B, int ldb, const float* SB, const float* bias, int act, int gated,
               int type, void* C, int ldc, hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || K > kMaxI8K) return GEMM_STATUS_INVALID_VALUE;
  if (!ld_ok(lda, K) || !ld_ok(ldb, K) || !ld_ok(ldc, N)) return GEMM_STATUS_INVALID_VALUE;
  if (!act_ok(act) || !float_type(type) || !flag_ok(gated)) return GEMM_STATUS_INVALID_VALUE;
  if (gated && N > (1 << 30)) return GEMM_STATUS_INVALID_VALUE;
  if (grouped) {
    if (groups < 0 || groups > kMaxExperts || per < 1 || a_rows < 0)
      return GEMM_STATUS_INVALID_VALUE;
    if (index == nullptr && a_rows < M) return GEMM_STATUS_INVALID_VALUE;
  }
  const bool empty = M == 0 || N == 0 || (grouped && groups == 0);
  const bool reads_ab = !empty && K > 0 && alpha != 0.0f;
  if (!empty && (C == nullptr || (grouped && offsets == nullptr))) return GEMM_STATUS_INVALID_VALUE;
  if (reads_ab && (A == nullptr || B == nullptr || SA == nullptr || SB == nullptr || a_rows == 0))
    return GEMM_STATUS_INVALID_VALUE;
  if (!aligned(C, elem(type)) || !aligned(SA, 4) || !aligned(SB, 4) || !aligned(bias, 4) ||
      !aligned(offsets, 4) || !aligned(index, 4))
    return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (empty) return GEMM_STATUS_SUCCESS;
  int alpha_e = 0;
  if (std::isfinite(alpha) && alpha != 0.0f) {
    alpha = 2.0f * std::frexp(alpha, &alpha_e);
    --alpha_e;
  }
  const lasg::I8Call c{M, N, reads_ab ? K : 0, alpha, A, lda, SA, reads_ab ? index : nullptr,
                       a_rows, per, B, ldb, alpha_e, SB, bias, act, gated, type, C, ldc, groups,
                       offsets};
  return finish(lasg::launch_i8_gemm(c, lasg::library_cus(), g_force_i8_tile.load(), stream));
}

// What the three calls that go token by token share; `rows`: of the sorted array.
bool exchange_ok(int tokens, int top_k, int cols, int type, int rows, const int* pos, const float* w) {
  return tokens >= 0 && top_k >= 1 && top_k <= kMaxTopK && cols >= 0 && float_type(type) &&
         rows >= 0 && aligned(pos, 4) && aligned(w, 4) &&
         (tokens == 0 || cols == 0 || pos != nullptr);
}

}  // namespace

extern "C" {

int i8_gemm_bias_act(int M, int N, int K, float alpha, const int8_t* A, int lda, const float* SA,
                     const int8_t* B, int ldb, const float* SB, const float* bias, int act, int gated,
                     int type, void* C, int ldc, hipStream_t stream) {
  return i8_product(false, 0, nullptr, M, N, K, alpha, A, lda, SA, M, nullptr, 1, B, ldb, SB, bias,
                    act, gated, type, C, ldc, stream);
}

int i8_gemm_grouped(int groups, const int* offsets, int M, int N, int K, float alpha, const int8_t* A,
                    int lda, const float* SA, int a_rows, const int* index, int per, const int8_t* B,
                    int ldb, const float* SB, const float* bias, int act, int gated, int type, void* C,
                    int ldc, hipStream_t stream) {
  return i8_product(true, groups, offsets, M, N, K, alpha, A, lda, SA, a_rows, index, per, B, ldb, SB,
                    bias, act, gated, type, C, ldc, stream);
}

int moe_sort_workspace(int tokens, int top_k, int experts, size_t* bytes) {
  if (tokens < 0 || top_k < 1 || top_k > kMaxTopK || experts < 1 || experts > kMaxExperts ||
      (int64_t)tokens * top_k > kMaxEntries || bytes == nullptr)
    return GEMM_STATUS_INVALID_VALUE;
  *bytes = lasg::sort_workspace_bytes((int64_t)tokens * top_k, experts);
  return GEMM_STATUS_SUCCESS;
}

int moe_sort(int tokens, int top_k, int experts, const int* ids, int* offsets, int* src, int* pos,
             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  if (moe_sort_workspace(tokens, top_k, experts, &need) != GEMM_STATUS_SUCCESS ||
      offsets == nullptr)
    return GEMM_STATUS_INVALID_VALUE;
  if (tokens > 0 && (ids == nullptr || src == nullptr || pos == nullptr || workspace == nullptr ||
                     workspace_bytes < need))
    return GEMM_STATUS_INVALID_VALUE;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(src, 4) || !aligned(pos, 4) ||
      !aligned(workspace, 256))
    return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  const lasg::SortCall c{tokens * top_k, experts, ids, offsets, src, pos, workspace};
  return finish(lasg::launch_sort(c, stream));
}

int moe_dispatch(int tokens, int top_k, int cols, int type, const void* X, int ldx, const int* pos,
                 const float* w, void* Y, int ldy, int y_rows, hipStream_t stream) {
  if (!exchange_ok(tokens, top_k, cols, type, y_rows, pos, w) || !ld_ok(ldx, cols) ||
      !ld_ok(ldy, cols) || !aligned(X, elem(type)) || !aligned(Y, elem(type)))
    return GEMM_STATUS_INVALID_VALUE;
  const bool empty = tokens == 0 || cols == 0 || y_rows == 0;
  if (!empty && (X == nullptr || Y == nullptr)) return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (empty) return GEMM_STATUS_SUCCESS;
  const lasg::ExchangeCall c{tokens, top_k, cols, type, X, ldx, nullptr, 0, y_rows, pos, w, Y, ldy,
                             nullptr};
  return finish(lasg::launch_dispatch(c, stream));
}

int moe_combine(int tokens, int top_k, int cols, int type, const void* X, int ldx, int x_rows,
                const int* pos, const float* w, void* Y, int ldy, hipStream_t stream) {
  if (!exchange_ok(tokens, top_k, cols, type, x_rows, pos, w) || !ld_ok(ldx, cols) ||
      !ld_ok(ldy, cols) || !aligned(X, elem(type)) || !aligned(Y, elem(type)))
    return GEMM_STATUS_INVALID_VALUE;
  const bool empty = tokens == 0 || cols == 0;
  if (!empty && ((X == nullptr && x_rows > 0) || Y == nullptr)) return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  if (empty) return GEMM_STATUS_SUCCESS;
  const lasg::ExchangeCall c{tokens, top_k, cols, type, nullptr, 0, X, ldx, x_rows, pos, w, Y, ldy,
                             nullptr};
  return finish(lasg::launch_combine(c, stream));
}

int moe_combine_grad(int tokens, int top_k, int cols, int type, const void* dY, int lddy,
                     const void* X, int ldx, int x_rows, const int* pos, const float* w, void* dX,
                     int lddx, float* dw, hipStream_t stream) {
  if (!exchange_ok(tokens, top_k, cols, type, x_rows, pos, w) || !ld_ok(lddy, cols) ||
      !aligned(dY, elem(type)) || !aligned(X, elem(type)) || !aligned(dX, elem(type)) ||
      !aligned(dw, 4))
    return GEMM_STATUS_INVALID_VALUE;
  if ((dw != nullptr && !ld_ok(ldx, cols)) || (dX != nullptr && !ld_ok(lddx, cols)))
    return GEMM_STATUS_INVALID_VALUE;
  if (tokens > 0 && dX == nullptr && dw == nullptr) return GEMM_STATUS_INVALID_VALUE;
  if (tokens > 0 && pos == nullptr) return GEMM_STATUS_INVALID_VALUE;
  const bool rows = tokens > 0 && cols > 0 && x_rows > 0;
  if (rows && (dY == nullptr || (dw != nullptr && X == nullptr))) return GEMM_STATUS_INVALID_VALUE;
  if (!lasg::library_ready()) return GEMM_STATUS_NOT_INITIALIZED;
  // Without columns or sorted rows there is no dX, dw is all zeros, and dY and X, which may be null
  // then, are not read: the kernel sees a call without columns.
  if (tokens == 0 || (!rows && dw == nullptr)) return GEMM_STATUS_SUCCESS;
  const lasg::ExchangeCall c{tokens, top_k, rows ? cols : 0, type, dY, lddy, X, ldx,
                             rows ? x_rows : 0, pos, w, dX, lddx, dw};
  return finish(lasg::launch_combine_grad(c, stream));
}

int gemm_debug_force_i8_tile(int tile) {
  if (tile < -1 || tile >= lasg::kI8TileCount) return GEMM_STATUS_INVALID_VALUE;
  g_force_i8_tile.store(tile);
  return GEMM_STATUS_SUCCESS;
}

int gemm_debug_force_moe_rows(int rows) {
  if (rows != 0 && rows != 16 && rows != 32 && rows != 64) return GEMM_STATUS_INVALID_VALUE;
  g_force_moe_rows.store(rows);
  return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
