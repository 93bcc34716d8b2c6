/*
 * gemm.h -- C ABI of the MI355X (gfx950) dense matrix-multiply library.
 *
 * The operation is the one stated in "SGEMM优化，从naive到warptiling",
 * section 问题与估算: C = alpha * A x B + beta * C, with A of M x K, B of K x N
 * and C of M x N, all row-major single-precision matrices.  The page's naive
 * kernel (section k1) takes (M, N, K, alpha, A, B, beta, C); this interface adds
 * leading dimensions and a HIP stream.  The half-precision entry point is the
 * FP16-input / FP32-accumulate product with bias and activation fused into the
 * single write-back, as described on the DeepGEMM page (sections 1.1 and 3.2).
 *
 * Conventions shared by every call:
 *  - Layout: row-major.  Element (i, j) of A is A[i*lda + j]; lda >= max(1, K),
 *    ldb >= max(1, N), ldc >= max(1, N).  No transpose options.
 *  - Memory: A, B, C and bias are DEVICE pointers owned by the caller; the
 *    library keeps no pointer after the enqueued work completes and allocates
 *    no device memory on the call path.  C must not overlap A, B or bias.
 *  - Alignment: element alignment only (4 bytes for float, 2 for half).
 *    Aligned shapes take a faster internal path; results do not depend on it.
 *  - Asynchrony: each call only enqueues work on `stream` (NULL = the default
 *    stream) and returns.  GEMM_STATUS_SUCCESS means "launched"; a device fault
 *    surfaces at the caller's next synchronisation.
 *  - Errors: invalid arguments return GEMM_STATUS_INVALID_VALUE and enqueue
 *    nothing (they are checked before anything else, with no HIP call).  A call
 *    before gemm_create returns GEMM_STATUS_NOT_INITIALIZED.  A failed launch
 *    returns GEMM_STATUS_HIP_ERROR; gemm_status_string then names the HIP error.
 *  - Threads: after gemm_create the compute calls may be made concurrently from
 *    several host threads and on several streams.  gemm_create/gemm_destroy must
 *    not race with compute calls.  Calls that use the library's workspace or pack
 *    buffer (split-K, operand copies) are ordered by the library: on one stream by
 *    stream order; the first such call on a second stream waits on the host for
 *    the device to finish its queued work (once), and from then on such calls
 *    order themselves with an event.  A call made while its stream is being
 *    captured into a HIP graph uses neither: it runs without split-K, and
 *    operands whose rows are off 16-byte boundaries are read in place by the
 *    bounds-checked kernels, so its replays need no ordering with other calls.
 */
#ifndef LINEAR_ALGEBRA_SGEMM_AMD_GEMM_H
#define LINEAR_ALGEBRA_SGEMM_AMD_GEMM_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GEMM_STATUS_SUCCESS = 0,
  GEMM_STATUS_NOT_INITIALIZED = 1,
  GEMM_STATUS_INVALID_VALUE = 2,
  GEMM_STATUS_ARCH_MISMATCH = 3,
  GEMM_STATUS_HIP_ERROR = 4,
  GEMM_STATUS_INTERNAL = 5
} gemm_status_t;

typedef enum {
  GEMM_ACT_NONE = 0,      /* identity */
  GEMM_ACT_GELU_TANH = 1, /* 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
  GEMM_ACT_SILU = 2       /* x / (1 + exp(-x)): the 8-bit products and moe_ffn only */
} gemm_act_t;

/* Element types of the 8-bit operators and the moe_ calls.  E4M3 is the 8-bit format
 * of 4 exponent and 3 mantissa bits with a NaN (bit patterns 0x7f, 0xff), no
 * infinity and the largest value 448. */
typedef enum {
  GEMM_TYPE_F32 = 0,
  GEMM_TYPE_F16 = 1,
  GEMM_TYPE_BF16 = 2,
  GEMM_TYPE_E4M3 = 3
} gemm_type_t;

/*
 * Initialise the library for the current HIP device.  Checks that the device
 * is gfx950 (else GEMM_STATUS_ARCH_MISMATCH) and records its compute-unit count.
 * Allocates the library's device memory: a 64 MiB workspace for split-K
 * partial sums and a 256 MiB buffer for packed copies of operands whose rows
 * do not start on 16-byte boundaries (a call may copy such an operand there,
 * with padded rows, so that its fastest kernels can read it).
 * Reference counted: each successful gemm_create needs one gemm_destroy.
 */
int gemm_create(void);

/* Drop one reference; the last one releases the library state.  The caller
 * synchronises its streams first.  Returns NOT_INITIALIZED if there is none. */
int gemm_destroy(void);

/*
 * C = alpha * A x B + beta * C in FP32 (section 问题与估算 of the SGEMM page),
 * computed with FP32 multiply-accumulate (MFMA, round to nearest even).
 *   M, N, K >= 0; A: M x K (lda), B: K x N (ldb), C: M x N (ldc), device pointers.
 *   beta == 0: C is write-only (NaN or Inf already in C does not propagate).
 *   alpha == 0 or K == 0: A and B are not read; C = beta * C.
 *   M == 0 or N == 0: nothing is done.
 * A null pointer is accepted only for an operand that is not read.
 */
int sgemm(int M, int N, int K, float alpha,
          const float* A, int lda, const float* B, int ldb,
          float beta, float* C, int ldc, hipStream_t stream);

/*
 * sgemm for callers that cannot allocate device memory on the call path: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, layout, conventions and errors as sgemm, and the
 * same kernels; it calls no hipMalloc, hipFree or allocating library routine.
 * Its split-K partial sums live in a static device array of 16 MiB (4 Mi
 * floats; one copy per GPU, held until the process ends) instead of the
 * workspace gemm_create allocates: split counts are limited to
 * splits * M * N <= 4 Mi, and operands whose rows are off 16-byte boundaries
 * are read by the bounds-checked kernels instead of being copied.  A plan that
 * would need more scratch returns GEMM_STATUS_INVALID_VALUE.  Needs
 * gemm_create, which looks the array up on its device (another device's is
 * looked up by the first call there).  Every sgemm_noalloc call on one GPU
 * shares that GPU's array, which keeps the last call's contents; calls that
 * overlap on one GPU (different streams, or a graph replayed while another
 * call runs) race.
 */
int sgemm_noalloc(int M, int N, int K, float alpha,
                  const float* A, int lda, const float* B, int ldb,
                  float beta, float* C, int ldc, hipStream_t stream);

/*
 * C = act(alpha * A x B + bias) with A (M x K) and B (K x N) in IEEE binary16
 * (passed as uint16_t bit patterns), FP32 accumulation, an FP32 bias of length
 * N added to every row (NULL = no bias), the activation `act` (gemm_act_t) and
 * C written as binary16, rounded to nearest even.  This is the fused epilogue
 * of the DeepGEMM page: bias, scale and activation applied in registers before
 * one store.  alpha == 0 or K == 0: A and B are not read.
 */
int hgemm_bias_act(int M, int N, int K, float alpha,
                   const uint16_t* A, int lda, const uint16_t* B, int ldb,
                   const float* bias, int act,
                   uint16_t* C, int ldc, hipStream_t stream);

/*
 * The same product with bfloat16 inputs and output (the upper 16 bits of an
 * IEEE binary32, passed as uint16_t bit patterns): C = act(alpha * A x B +
 * bias), FP32 accumulation, C rounded to nearest even.  Arguments, layout,
 * conventions and errors are those of hgemm_bias_act.
 */
int bgemm_bias_act(int M, int N, int K, float alpha,
                   const uint16_t* A, int lda, const uint16_t* B, int ldb,
                   const float* bias, int act,
                   uint16_t* C, int ldc, hipStream_t stream);

/*
 * Block quantisation to e4m3.  With s = max(max|x| / 448, 2^-126) over a block
 * of `block_rows` (1 or 128) rows and 128 columns of X (rows x cols, `type`
 * F32, F16 or BF16; the last blocks of a row or column may be shorter),
 *   Q[i][j] = x[i][j] / s, rounded to e4m3 to nearest even,
 *   S[j / 128][i] = s  (block_rows 1)  or  S[j / 128][i / 128] = s  (128),
 * s and x / s rounded to fp32 for 16-bit X; for FP32 X the quotient is by s before
 * it is rounded.  (A quotient that is a tie in exact arithmetic may go to either
 * neighbour with a rounded s: a bfloat16 x = 2.90625 in a block with max|x| = 62
 * gives 22, where 448 x / 62 is 21, a tie that even takes to 20.)
 * Q rows x cols with leading dimension ldq >= cols, S with lds >= rows, or >=
 * ceil(rows / 128).  QT, ST: the same of the transpose of X: QT cols x rows
 * (ldqt >= rows), blocks of 128 rows of X by one column (ST[i / 128][j]) or by
 * 128 (ST[i / 128][j / 128]), ldst >= cols or ceil(cols / 128).  Q with S, or
 * QT with ST, may be null (their leading dimensions are then ignored), not
 * both pairs.  A block that holds a NaN has a NaN scale and NaN values; one that holds an
 * infinity an infinite scale, NaN for its infinities and 0 for the rest.
 * rows == 0 or cols == 0: nothing is done.
 */
int fp8_quantize(int rows, int cols, int type, const void* X, int ldx, int block_rows,
                 uint8_t* Q, int ldq, float* S, int lds,
                 uint8_t* QT, int ldqt, float* ST, int ldst, hipStream_t stream);

/*
 * The block-scaled e4m3 product with fused bias and activation,
 *   C[m][n] = act(alpha sum_k SA[k / 128][m] A[m][k] SB[k / 128][n / b_rows] B[n][k] + bias[n]),
 * A M x K (lda >= K) and B N x K (ldb >= K; the transposed operand, as
 * fp8_quantize's outputs are laid out), ldsa >= M, b_rows 1 or 128 with ldsb >=
 * N or ceil(N / 128), an FP32 bias of length N (NULL = none), `act` of
 * gemm_act_t, C of `type` F32, F16 or BF16, rounded once to nearest even.
 * Bytes of A and B past column K are not used.  alpha == 0 or K == 0: A, B and
 * the scales are not read.
 * A block's two scales are multiplied with each other first, in fp32.  Where their
 * product is below 2^-126 (as of a zero row's scale, 2^-126, with most others) the
 * block's term, itself below 2^-101, is off by up to 2^-125; where it passes
 * fp32's range the term is infinite, or NaN if the block's sum is 0.
 * fast_sums 0: each block's sum is formed in fp32 from exact products.
 * fast_sums 1: by the 8-bit matrix instructions, at twice the rate; they add
 * eight consecutive columns at a time and drop, of each product, what lies below
 * 2^-13 of the largest one's power of two.  At worst, one column far above the
 * seven beside it, that is 7 / 2^13 = 8.6e-4 of sum_k |a||b| (eight times that where
 * the largest product is of a value below 2^-6, which counts as 2^-6 there); 1e-5
 * was measured for data of one magnitude, 2e-4 for magnitudes over several
 * powers of ten: meant for 16-bit results.  The sums over blocks are fp32 either way.
 */
int fp8_gemm_bias_act(int M, int N, int K, float alpha,
                      const uint8_t* A, int lda, const float* SA, int ldsa,
                      const uint8_t* B, int ldb, const float* SB, int ldsb, int b_rows,
                      const float* bias, int act, int type, void* C, int ldc,
                      int fast_sums, hipStream_t stream);

/* A mixture-of-experts feed-forward layer (moe_ffn). */
typedef struct {
  int tokens;       /* T, 0 .. 64 */
  int d_model;      /* D, 1 .. 2^20 */
  int d_ff;         /* I, 1 .. 2^20 */
  int experts;      /* E, 1 .. 1024 */
  int top_k;        /* k, 1 .. min(E, 32) */
  int type;         /* of X, R and Y: F16 or BF16 */
  int weight_type;  /* of W1 and W2: `type` or E4M3 */
  int act;          /* gemm_act_t */
  int gated;        /* 1: W1 has 2 I rows, and act(first I) multiplies the second I */
  int norm_topk;    /* 1: a token's k weights are divided by their sum */
} moe_shape_t;

/* Bytes of device memory a moe_ffn call of this shape needs as `workspace`. */
int moe_ffn_workspace(const moe_shape_t* shape, size_t* bytes);

/*
 * The layer, for the few tokens of a decoding step.  (More tokens, with int8 weights and with
 * experts and weights of the caller's own router: moe_sort, i8_gemm_grouped, moe_combine.)
 *   l = X R^T (T x E),  ids[t] = the k largest of l[t], largest first, equal
 *   ones by lower number,  w[t] = softmax(l[t]) at ids[t] (divided by their sum
 *   with norm_topk),  Y[t] = sum_s w[t][s] W2[e] h(W1[e] X[t]),  e = ids[t][s],
 *   h(u) = act(u), or with `gated` act(u[0 .. I)) u[I .. 2 I).
 * X T x D (ldx), R E x D (ldr), W1 E matrices of (gated ? 2 I : I) x D (ld1)
 * one behind the other, W2 E matrices of D x I (ld2), ids (int32) and w (FP32)
 * T x k dense, Y T x D (ldy).  With E4M3 weights S1 and S2 hold a scale for every 128 x
 * 128 block of each matrix, expert by expert, column block by column block:
 * S1[e][d / 128][row / 128], S2[e][i / 128][d / 128], dense; else they are
 * ignored.  Columns past D or I of a row are not used.
 * The logits and the choice are computed in 64 bits, products with fp32 sums;
 * h is kept as two numbers of `type`: in BF16 to 2^-17 of itself, in F16 to 2^-17
 * of a token's largest |h| for that expert or better, and in F16 its range is
 * +-65504 (larger finite values are clamped to that).
 * `workspace` (256-byte aligned, at least moe_ffn_workspace bytes) belongs to
 * the call until its work on `stream` is done; its contents need no
 * preparation.  tokens == 0: nothing is done.
 */
int moe_ffn(const moe_shape_t* shape, const uint16_t* X, int ldx, const uint16_t* R, int ldr,
            const void* W1, int ld1, const float* S1, const void* W2, int ld2, const float* S2,
            int* ids, float* w, uint16_t* Y, int ldy, void* workspace, size_t workspace_bytes,
            hipStream_t stream);

/*
 * Quantisation of rows to int8: with s = max(max|x| / 127, 2^-126) over row r of X
 * (rows x cols, `type` F32, F16 or BF16, cols at most 2^20),
 *   Q[r][j] = x[r][j] / s, rounded to the nearest whole number, ties to even,
 *   S[r] = s,
 * s and x / s rounded to fp32.  Tokens and the channels of a weight (one a row) are
 * quantised alike.  Q rows x cols with ldq >= cols; S dense.  A row that holds a NaN or an
 * infinity has that for its scale and zeros for its values, so that its products
 * are NaN.  rows == 0 or cols == 0: nothing is done.
 */
int i8_quantize(int rows, int cols, int type, const void* X, int ldx,
                int8_t* Q, int ldq, float* S, hipStream_t stream);

/*
 * The int8 product with a scale for every token and channel,
 *   u[m][n] = alpha SA[m] SB[n] sum_k A[m][k] B[n][k] + bias[n],
 *   C[m][n] = act(u[m][n]),  or with gated 1  act(u[m][n]) u[m][N + n],
 * A M x K (lda >= K), B N x K, with a gate 2 N x K (ldb >= K; one channel a row, as
 * i8_quantize lays it out), SA of length M, SB and bias (FP32, NULL = none) one value for
 * every row of B, `act` of gemm_act_t, C (ldc >= N) of `type` F32, F16 or BF16, rounded
 * once to nearest even.  K is at most 131071: the sums are exact, in int32, and are
 * rounded to fp32 once before they are scaled.  All values of int8 may occur, -128
 * too.  Bytes of A and B past column K are not used.  alpha, the scales and the sum are
 * multiplied without a detour past fp32's range: only their product has to be inside it.  alpha == 0 or
 * K == 0: A, B and the scales are not read.  With a gate N is at most 2^30.
 * (Where M times the rows of B pass about 2^34, or either passes 2^30, a result takes some seven
 * times as long.)
 */
int i8_gemm_bias_act(int M, int N, int K, float alpha,
                     const int8_t* A, int lda, const float* SA,
                     const int8_t* B, int ldb, const float* SB,
                     const float* bias, int act, int gated, int type, void* C, int ldc,
                     hipStream_t stream);

/*
 * The same product of `groups` (at most 1024) sets of rows, each with a matrix of its own, as
 * the experts of a layer take their tokens.  Row r, offsets[g] <= r < offsets[g + 1] (device
 * memory, groups + 1 int32 numbers that ascend, as moe_sort writes them; the rows
 * number at most M), is multiplied by group g's matrix: B, SB and bias hold the groups' one
 * behind the other (N rows each, 2 N with a gate).  Rows outside every group are
 * left as they were in C (M rows of it).
 * `index` NULL: row r of the product is row r of A (a_rows >= M).  Else it is row
 * index[r] / per of A and SA, which have a_rows rows: with moe_sort's src and per = top_k
 * tokens are read where they lie.  (A row number past the end is taken as the last row of A, a
 * negative one as row 0; offsets that do not ascend give unspecified results, but no
 * access outside the arrays.)
 */
int i8_gemm_grouped(int groups, const int* offsets, int M, int N, int K, float alpha,
                    const int8_t* A, int lda, const float* SA, int a_rows,
                    const int* index, int per,
                    const int8_t* B, int ldb, const float* SB,
                    const float* bias, int act, int gated, int type, void* C, int ldc,
                    hipStream_t stream);

/* Bytes of device memory a moe_sort call of this shape needs as `workspace`. */
int moe_sort_workspace(int tokens, int top_k, int experts, size_t* bytes);

/*
 * Tokens in the order of their experts: a stable sort of ids (tokens x top_k dense, the expert
 * of every token's slots; numbers outside 0 .. experts - 1 are no expert's, as those of padding).
 *   offsets[e] (experts + 1)       the first row of expert e; offsets[experts] rows in all,
 *   src[row] (tokens x top_k)      the entry token * top_k + slot of every row, -1 behind the last,
 *   pos[token][slot] (as ids)      the row of every entry, -1 for those of no expert.
 * An expert's rows are in the order of their entries.  experts 1 .. 1024, top_k 1 .. 32,
 * tokens x top_k at most 2^30; a token may name an expert twice.  `workspace` (256-byte
 * aligned, at least moe_sort_workspace bytes) belongs to the call until its work on `stream`
 * is done; its contents need no preparation.
 */
int moe_sort(int tokens, int top_k, int experts, const int* ids, int* offsets, int* src, int* pos,
             void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Tokens into sorted rows: Y[pos[t][s]] = X[t], times w[t][s] where w (FP32, tokens x top_k dense) is
 * not NULL.  X tokens x cols (ldx), Y y_rows x cols (ldy), both of `type` F32, F16 or BF16;
 * products fp32, rounded once.  Entries of pos outside 0 .. y_rows - 1 are
 * skipped; rows of Y that none names are left as they were, and no two may name the same.
 * Gradients: to X that is moe_combine of Y's gradient with the same pos and w, to w
 * moe_combine_grad's dw with X for its dY and Y's gradient for its X.
 */
int moe_dispatch(int tokens, int top_k, int cols, int type, const void* X, int ldx,
                 const int* pos, const float* w, void* Y, int ldy, int y_rows, hipStream_t stream);

/*
 * Sorted rows back to their tokens: Y[t] = sum_s w[t][s] X[pos[t][s]] (w NULL: ones), fp32 sums in the
 * order of the slots, rounded once.  X x_rows x cols (ldx), Y tokens x cols (ldy).  Entries of
 * pos outside 0 .. x_rows - 1 are skipped (whatever their w); a token without any is zero.
 */
int moe_combine(int tokens, int top_k, int cols, int type, const void* X, int ldx, int x_rows,
                const int* pos, const float* w, void* Y, int ldy, hipStream_t stream);

/*
 * moe_combine's gradients:
 *   dX[pos[t][s]] = w[t][s] dY[t],   dw[t][s] = sum_c dY[t][c] X[pos[t][s]][c],
 * dw FP32 (tokens x top_k dense), 0 for entries outside 0 .. x_rows - 1; dX x_rows x cols (lddx), of
 * which rows that no entry names are left as they were, and no two may name the same.  Either dX
 * or dw may be NULL: then it is not wanted (without dw X is not read).  dX must not
 * overlap X or dY.  x_rows == 0 or cols == 0: dw is all zeros, and dY, X and dX are not touched.
 */
int moe_combine_grad(int tokens, int top_k, int cols, int type, const void* dY, int lddy,
                     const void* X, int ldx, int x_rows, const int* pos, const float* w,
                     void* dX, int lddx, float* dw, hipStream_t stream);

/* Static text for a status code; for GEMM_STATUS_HIP_ERROR it also names the
 * last HIP error seen by the library on this host thread. */
const char* gemm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_ALGEBRA_SGEMM_AMD_GEMM_H */
