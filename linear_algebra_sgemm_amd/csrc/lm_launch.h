// Internal interface between the C ABI of the 8-bit operators and the
// mixture-of-experts layer (lm_capi.cpp) and their kernels.  Arguments arrive
// here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gemm.h"

namespace lasg {

// Library state (gemm_capi.cpp): whether gemm_create has run, the compute units
// of its device, and the status of a failed HIP call (kept for
// gemm_status_string).
bool library_ready();
int library_cus();
int library_hip_failure(hipError_t e);
int library_force_fp8_tile();   // gemm_debug_force_tile(2, ...)

struct QuantizeCall {
  int rows, cols, type;
  const void* X;
  int ldx;
  int block_rows;   // 1 or 128
  uint8_t* Q;       // null: not wanted
  int ldq;
  float* S;
  int lds;
  uint8_t* QT;      // null: not wanted
  int ldqt;
  float* ST;
  int ldst;
};
hipError_t launch_quantize(const QuantizeCall& c, hipStream_t s);

struct Fp8Call {
  int M, N, K;      // K == 0: the product is zero and A, B are not read
  float alpha;
  const uint8_t* A;
  int lda;
  const float* SA;
  int ldsa;
  const uint8_t* B;
  int ldb;
  const float* SB;
  int ldsb;
  int b_rows;       // rows of B that share a scale: 1 or 128
  const float* bias;
  int act;
  int type;         // of C
  void* C;
  int ldc;
  bool fast_sums;
};
// Output tile: 0 = 128 x 256 (fast sums and one scale per 128 rows of B only), 1 =
// 128 x 128, 2 = 64 x 64 with four stages of LDS, 3 = with three, copied straight
// into LDS; 4 = 128 x 128 for other operands; with K split over a workgroup's
// waves 5 = 64 x 32, 6 = 64 x 16, 7 = 32 x 32, 8 = 32 x 16, 9 = 16 x 32 and 10 = 16 x 16.
constexpr int kFp8TileCount = 11;
// The tile that runs for a call on `cus` compute units: `force`, or by shape
// where that is -1; resolved to one that applies.
int fp8_tile(const Fp8Call& c, int cus, int force);
hipError_t launch_fp8_gemm(const Fp8Call& c, int cus, int force, hipStream_t s);

struct MoeCall {
  moe_shape_t shape;
  const uint16_t* X;
  int ldx;
  const uint16_t* R;
  int ldr;
  const void* W1;
  int ld1;
  const float* S1;
  const void* W2;
  int ld2;
  const float* S2;
  int* ids;
  float* w;
  uint16_t* Y;
  int ldy;
  void* ws;
};
size_t moe_workspace_bytes(const moe_shape_t& s);
// `force_rows`: rows of a weight per workgroup, 0 = by shape.
hipError_t launch_moe(const MoeCall& c, int cus, int force_rows, hipStream_t s);

struct I8QuantizeCall {
  int rows, cols, type;
  const void* X;
  int ldx;
  int8_t* Q;
  int ldq;
  float* S;
};
hipError_t launch_i8_quantize(const I8QuantizeCall& c, int cus, hipStream_t s);

struct I8Call {
  int M, N, K;      // K == 0: the sums are zero; A, B and their scales are not read
  float alpha;      // the caller's is alpha 2^alpha_e, 1 <= |alpha| < 2 where it is finite and not 0
  const int8_t* A;
  int lda;
  const float* SA;
  const int* index; // null, or row r of the product reads row index[r] / per of A
  int a_rows, per;
  const int8_t* B;  // a group's matrix behind the other, SB and bias likewise
  int ldb;
  // (In a gap of the struct, and in this one: beside alpha or type the 16-row K-split kernels loaded their
  // arguments in one more dependent step, 6.2 us for one token by 4096 x 4096 in place of 6.05.)
  int alpha_e;
  const float* SB;
  const float* bias;
  int act, gated;
  int type;         // of C
  void* C;
  int ldc;
  int groups;       // 0: one product of all rows
  const int* offsets;
};
// Output tile: 0 = 256 x 256, 1 = 128 x 256, 2 = 128 x 128, 3 = 64 x 128, 4 = 64 x 64 and 5 =
// 32 x 128 copied straight into LDS; 6 = 128 x 128 through registers; with K split over a
// workgroup's waves 7 = 64 x 32, 8 = 32 x 32, 9 = 32 x 16, 10 = 16 x 32, 11 = 16 x 16.  (Columns are
// rows of B: half as many of C with a gate.)
constexpr int kI8TileCount = 12;
int i8_tile(const I8Call& c, int cus, int force);
hipError_t launch_i8_gemm(const I8Call& c, int cus, int force, hipStream_t s);

// Tokens in the experts' order and back (exchange_kernels.hip).
struct SortCall {
  int entries, experts;
  const int* ids;
  int* offsets;
  int* src;
  int* pos;
  void* ws;
};
size_t sort_workspace_bytes(int64_t entries, int experts);
hipError_t launch_sort(const SortCall& c, hipStream_t s);

struct ExchangeCall {
  int tokens, top_k, cols, type;
  const void* tok;      // one row a token (dispatch's X, the gradient's dY); null for combine
  int ldtok;
  const void* sorted;   // one row a (token, slot), in the experts' order; null for dispatch
  int ldsorted;
  int rows;             // of the sorted arrays
  const int* pos;
  const float* w;       // null: ones
  void* out;            // dispatch's and the gradient's sorted rows, combine's tokens
  int ldout;
  float* dw;            // the gradient's
};
hipError_t launch_dispatch(const ExchangeCall& c, hipStream_t s);
hipError_t launch_combine(const ExchangeCall& c, hipStream_t s);
hipError_t launch_combine_grad(const ExchangeCall& c, hipStream_t s);

}  // namespace lasg
