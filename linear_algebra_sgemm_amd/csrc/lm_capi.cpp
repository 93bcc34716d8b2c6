// C ABI of the 8-bit operators and the mixture-of-experts layer (declared in
// include/gemm.h): argument checks, quick returns, and the launch.  None of
// these calls allocates, copies to the host or uses the library's own
// workspace, so all may be captured into a graph and run on any stream.
#include <atomic>

#include "../../include/gemm_debug.h"
#include "lm_launch.h"

namespace {

std::atomic<int> g_force_moe_rows{0};

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

int gemm_debug_force_moe_rows(int rows) {
  if (rows != 0 && rows != 16 && rows != 32 && rows != 64) return GEMM_STATUS_INVALID_VALUE;
  g_force_moe_rows.store(rows);
  return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
