// A mixture-of-experts feed-forward layer for a few tokens (at most 64):
//     l[t][e]  = sum_d X[t][d] R[e][d]
//     ids[t]   = the top_k largest l[t], largest first, ties to the lower expert
//     w[t]     = softmax(l[t]) at ids[t], divided by their sum if asked for
//     h[t][s]  = act(W1[e] x) (* the second half of W1's rows when gated), e = ids[t][s]
//     Y[t]     = sum_s w[t][s] W2[e] h[t][s]
//
// What bounds it are the chosen experts' weights, each of which is read once:
// the tokens that chose an expert form the rows of one small product against
// it.  A workgroup takes an expert and 16 rows of its weight; its eight waves
// split the columns, read the weight straight into MFMA operands (16x16x32,
// the tokens as the other operand) and add their fp32 sums in LDS.  Which
// experts there are is known on the device only: the grid has a row for every
// (token, slot) pair or every expert, whichever is fewer, and workgroups whose
// expert another row takes, or nobody chose, end at once.
//
// The logits are summed in 64 bits: two experts' logits can lie closer than
// fp32 sums of a few thousand terms resolve, and the choice between them is an
// output.  The inner activations h are kept to about 16 (bfloat16) or 22
// (binary16) bits as a pair hi + lo of the 16-bit type, each multiplied by W2:
// rounded to one such number they would cost as much accuracy as the final
// rounding of Y, and the second MFMA is free beside the loads.  In binary16 hi
// is clamped to +-65504, the type's range.
#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

namespace {

constexpr int kMaxTokens = 64;   // one wave's lanes hold the tokens

// Where the parts of the workspace lie (bytes).
struct MoeWorkspace {
  size_t logits, h, part, bytes;
  int ldh;   // elements per row of h_hi, h_lo
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

MoeWorkspace moe_layout(const moe_shape_t& s) {
  MoeWorkspace w;
  const size_t pairs = (size_t)s.tokens * s.top_k;
  w.ldh = (int)(((size_t)s.d_ff + 127) / 128 * 128);
  w.logits = 0;
  w.h = round256((size_t)s.tokens * s.experts * sizeof(double));
  w.part = w.h + round256(2 * pairs * w.ldh * sizeof(uint16_t));
  w.bytes = w.part + round256(pairs * s.d_model * sizeof(float));
  return w;
}

struct MoeArgs {
  int tokens, d_model, d_ff, experts, top_k, act;
  bool norm, by_expert;   // by_expert: grid rows are experts, else pairs
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* R;
  int64_t ldr;
  const void* W1;
  int64_t ld1;
  const float* S1;
  const void* W2;
  int64_t ld2;
  const float* S2;
  int* ids;
  float* w;
  uint16_t* Y;
  int64_t ldy;
  double* logits;
  uint16_t* h_hi;
  uint16_t* h_lo;
  int64_t ldh;
  float* part;
};

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// The tokens that chose a grid row's expert, in token order: `pair[i]` is
// token * top_k + slot.  Lane t of every wave looks at token t.
struct Rows {
  int expert, count;   // count == 0: nothing for this workgroup
};
__device__ __forceinline__ Rows find_rows(const MoeArgs& p, int grid_row, int* pair) {
  const int lane = threadIdx.x % kWave;
  Rows out;
  out.expert = p.by_expert ? grid_row : p.ids[grid_row];
  int slot = -1;
  if (lane < p.tokens) {
    const int* ids = p.ids + lane * p.top_k;
    for (int s = 0; s < p.top_k; ++s)
      if (ids[s] == out.expert) slot = s;
  }
  const uint64_t mask = __ballot(slot >= 0);
  out.count = __popcll(mask);
  const int mine = lane * p.top_k + slot;
  if (!p.by_expert && out.count > 0) {
    // The pair of the first token that chose the expert does the work.
    const int first = __shfl(mine, __ffsll((unsigned long long)mask) - 1);
    if (first != grid_row) out.count = 0;
  }
  if (out.count == 0) return out;
  if (threadIdx.x < kWave && slot >= 0)
    pair[__popcll(mask & ((uint64_t(1) << lane) - 1))] = mine;
  __syncthreads();
  return out;
}

// 128 columns of 16 rows of a weight as the first operands of four MFMAs; the
// order of the columns depends on how the type is loaded (16 bytes a lane), and
// `column` gives the first of the eight that MFMA t of lane group g multiplies.
template <class E, bool FP8>
struct WeightBlock {
  typename E::vec8 v[4];
  static __device__ __forceinline__ int column(int t, int g) {
    return FP8 ? 64 * (t / 2) + 16 * g + 8 * (t % 2) : 32 * t + 8 * g;
  }
  // Columns k0 .. k0 + 127 of a row of `cols`.
  __device__ __forceinline__ void load(const void* row, int k0, int g, int cols) {
    const uint8_t* b = static_cast<const uint8_t*>(row);
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = k0 + 64 * u + 16 * g;
        const u32x4 c = cols - k0 >= kBlockK ? load16(b + at) : load16_row(b, at, cols);
        v[2 * u] = E::widen(c[0], c[1]);
        v[2 * u + 1] = E::widen(c[2], c[3]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int at = 2 * (k0 + column(t, g));
        v[t] = __builtin_bit_cast(typename E::vec8, cols - k0 >= kBlockK
                                                        ? load16(b + at)
                                                        : load16_row(b, at, 2 * cols));
      }
    }
  }
};

// Columns col .. col + 7 of a row of `cols`, in the block of 128 from k0.
template <class E>
__device__ __forceinline__ typename E::vec8 load_x(const uint16_t* row, int k0, int col, int cols) {
  return __builtin_bit_cast(typename E::vec8, cols - k0 >= kBlockK
                                                  ? load16(row + k0 + col)
                                                  : load16_row(row, 2 * (k0 + col), 2 * cols));
}

}  // namespace

// Logits of one expert and four tokens per workgroup, its four waves splitting
// the columns; products and sums in 64 bits.
template <class E>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeArgs p) {
  constexpr int TT = 4;
  __shared__ double sums[4][TT];
  const int e = blockIdx.x, t0 = TT * blockIdx.y;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const uint16_t* r = p.R + e * p.ldr;
  double acc[TT] = {};
  for (int d = 8 * threadIdx.x; d < p.d_model; d += 8 * 256) {
    const u32x4 rv = load8h_upto(r + d, p.d_model - d);
    double rd[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rd[i] = E::value((uint16_t)(rv[i / 2] >> (16 * (i % 2))));
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int token = t0 + t < p.tokens ? t0 + t : p.tokens - 1;
      const u32x4 xv = load8h_upto(p.X + token * p.ldx + d, p.d_model - d);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[t] = __builtin_fma((double)E::value((uint16_t)(xv[i / 2] >> (16 * (i % 2)))), rd[i],
                               acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const double s = wave_sum(acc[t]);
    if (lane == 0) sums[wave][t] = s;
  }
  __syncthreads();
  if (threadIdx.x < TT && t0 + (int)threadIdx.x < p.tokens) {
    const int t = threadIdx.x;
    p.logits[(int64_t)(t0 + t) * p.experts + e] = (sums[0][t] + sums[1][t]) + (sums[2][t] + sums[3][t]);
  }
}

// One wave per token: an expert's place is the number of experts before it in
// the order (NaN first, then larger logits, then lower numbers: a total order,
// so the places are a permutation whatever the logits are).
__global__ void __launch_bounds__(64) moe_route_kernel(MoeArgs p) {
  extern __shared__ double key[];   // experts
  __shared__ double chosen[kMaxTokens];   // by place, below top_k
  const int lane = threadIdx.x, t = blockIdx.x;
  double top = -__builtin_inf();
  for (int e = lane; e < p.experts; e += kWave) {
    key[e] = p.logits[(int64_t)t * p.experts + e];
    top = key[e] > top ? key[e] : top;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  __syncthreads();
  double sum = 0.0;
  for (int e = lane; e < p.experts; e += kWave) sum += exp(key[e] - top);
  sum = wave_sum(sum);
  for (int e = lane; e < p.experts; e += kWave) {
    const double v = key[e];
    int place = 0;
    for (int o = 0; o < p.experts; ++o) {
      const double u = key[o];
      const bool un = u != u, vn = v != v;
      const bool before = un || vn ? un && (!vn || o < e) : u > v || (u == v && o < e);
      place += before;
    }
    if (place < p.top_k) {
      p.ids[t * p.top_k + place] = e;
      chosen[place] = exp(v - top) / sum;
    }
  }
  __syncthreads();
  if (lane < p.top_k) {
    double total = 1.0;
    if (p.norm) {
      total = 0.0;
      for (int s = 0; s < p.top_k; ++s) total += chosen[s];
    }
    p.w[t * p.top_k + lane] = (float)(chosen[lane] / total);
  }
}

// h for 16 inner columns of one expert and all its tokens (at most 16 MF).
template <class E, bool FP8, bool GATED, int MF>
__global__ void __launch_bounds__(512) moe_up_kernel(MoeArgs p) {
  constexpr int SIDES = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float part[8][SIDES][MF][256];
  __shared__ int pair[kMaxTokens];
  const Rows rows = find_rows(p, blockIdx.y, pair);
  if (rows.count == 0) return;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, g = lane / 16;
  const int n0 = 16 * blockIdx.x;
  const int D = p.d_model, I = p.d_ff;
  const int64_t rows1 = (int64_t)SIDES * I;
  const uint16_t* x[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int at = 16 * i + r < rows.count ? 16 * i + r : rows.count - 1;
    x[i] = p.X + (int64_t)(pair[at] / p.top_k) * p.ldx;
  }
  const uint8_t* w[SIDES];
  const float* scale[SIDES][4];
  const int64_t rbs = (rows1 + 127) / 128;
  const int64_t kbs = (D + 127) / 128;
#pragma unroll
  for (int side = 0; side < SIDES; ++side) {
    const int n = n0 + r < I ? n0 + r : I - 1;   // (rows past the end: never stored)
    const int64_t row = (int64_t)rows.expert * rows1 + (int64_t)side * I + n;
    w[side] = static_cast<const uint8_t*>(p.W1) + row * p.ld1 * (FP8 ? 1 : 2);
    if constexpr (FP8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ne = n0 + 4 * g + e < I ? n0 + 4 * g + e : I - 1;
        scale[side][e] = p.S1 + (int64_t)rows.expert * kbs * rbs + ((int64_t)side * I + ne) / 128;
      }
    }
  }
  f32x4 total[SIDES][MF];
#pragma unroll
  for (int side = 0; side < SIDES; ++side)
#pragma unroll
    for (int i = 0; i < MF; ++i) total[side][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = wave; kb < kbs; kb += 8) {
    const int k0 = kb * kBlockK;
    WeightBlock<E, FP8> wb[SIDES];
#pragma unroll
    for (int side = 0; side < SIDES; ++side) wb[side].load(w[side], k0, g, D);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if (16 * i >= rows.count) break;
      f32x4 v[SIDES];
#pragma unroll
      for (int side = 0; side < SIDES; ++side)
        v[side] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : total[side][i];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const auto xv = load_x<E>(x[i], k0, WeightBlock<E, FP8>::column(t, g), D);
#pragma unroll
        for (int side = 0; side < SIDES; ++side) v[side] = E::mfma(wb[side].v[t], xv, v[side]);
      }
#pragma unroll
      for (int side = 0; side < SIDES; ++side) {
        if constexpr (FP8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            total[side][i][e] =
                __builtin_fmaf(v[side][e], scale[side][e][kb * rbs], total[side][i][e]);
        } else {
          total[side][i] = v[side];
        }
      }
    }
  }
#pragma unroll
  for (int side = 0; side < SIDES; ++side)
#pragma unroll
    for (int i = 0; i < MF; ++i)
      *reinterpret_cast<f32x4*>(&part[wave][side][i][4 * lane]) = total[side][i];
  __syncthreads();
  for (int v = threadIdx.x; v < MF * 256; v += 512) {
    const int i = v / 256, at = v % 256;
    const int token = 16 * i + (at / 4) % 16, n = n0 + 4 * (at / 64) + at % 4;
    if (token >= rows.count || n >= I) continue;
    float s[SIDES];
#pragma unroll
    for (int side = 0; side < SIDES; ++side) {
      s[side] = part[0][side][i][at];
#pragma unroll
      for (int q = 1; q < 8; ++q) s[side] += part[q][side][i][at];
    }
    float h = apply_act(s[0], p.act);
    if constexpr (GATED) h *= s[SIDES - 1];
    const bool inf = __builtin_fabsf(h) == __builtin_inff();   // (infinities and NaN stay)
    if (!inf) h = h > E::kMax ? E::kMax : h < -E::kMax ? -E::kMax : h;
    const uint16_t hi = E::bits(h);
    const int64_t at_h = (int64_t)pair[token] * p.ldh + n;
    p.h_hi[at_h] = hi;
    p.h_lo[at_h] = E::bits(inf ? 0.0f : h - E::value(hi));
  }
}

// w h W2 of 16 output columns of one expert and all its tokens, per pair.
template <class E, bool FP8, int MF>
__global__ void __launch_bounds__(512) moe_down_kernel(MoeArgs p) {
  __shared__ __attribute__((aligned(16))) float part[8][MF][256];
  __shared__ int pair[kMaxTokens];
  const Rows rows = find_rows(p, blockIdx.y, pair);
  if (rows.count == 0) return;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, g = lane / 16;
  const int n0 = 16 * blockIdx.x;
  const int D = p.d_model, I = p.d_ff;
  int64_t h_row[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int at = 16 * i + r < rows.count ? 16 * i + r : rows.count - 1;
    h_row[i] = pair[at] * p.ldh;
  }
  const int n = n0 + r < D ? n0 + r : D - 1;
  const uint8_t* w = static_cast<const uint8_t*>(p.W2) +
                     ((int64_t)rows.expert * D + n) * p.ld2 * (FP8 ? 1 : 2);
  const int64_t rbs = (D + 127) / 128;
  const int64_t kbs = (I + 127) / 128;
  const float* scale = FP8 ? p.S2 + rows.expert * kbs * rbs + n0 / 128 : nullptr;
  f32x4 total[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) total[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = wave; kb < kbs; kb += 8) {
    const int k0 = kb * kBlockK;
    WeightBlock<E, FP8> wb;
    wb.load(w, k0, g, I);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if (16 * i >= rows.count) break;
      f32x4 v = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : total[i];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int col = WeightBlock<E, FP8>::column(t, g);
        v = E::mfma(wb.v[t], load_x<E>(p.h_hi + h_row[i], k0, col, I), v);
        v = E::mfma(wb.v[t], load_x<E>(p.h_lo + h_row[i], k0, col, I), v);
      }
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          total[i][e] = __builtin_fmaf(v[e], scale[kb * rbs], total[i][e]);
      } else {
        total[i] = v;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) *reinterpret_cast<f32x4*>(&part[wave][i][4 * lane]) = total[i];
  __syncthreads();
  for (int v = threadIdx.x; v < MF * 256; v += 512) {
    const int i = v / 256, at = v % 256;
    const int token = 16 * i + (at / 4) % 16, col = n0 + 4 * (at / 64) + at % 4;
    if (token >= rows.count || col >= D) continue;
    float s = part[0][i][at];
#pragma unroll
    for (int q = 1; q < 8; ++q) s += part[q][i][at];
    p.part[(int64_t)pair[token] * D + col] = p.w[pair[token]] * s;
  }
}

// The slots of a token added in their order (no atomics: the same bits every time).
template <class E>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeArgs p) {
  const int t = blockIdx.y;
  for (int d = blockIdx.x * 256 + threadIdx.x; d < p.d_model; d += gridDim.x * 256) {
    float s = 0.0f;
    for (int q = 0; q < p.top_k; ++q)
      s += p.part[((int64_t)t * p.top_k + q) * p.d_model + d];
    p.Y[t * p.ldy + d] = E::bits(s);
  }
}

namespace {

template <class E, bool FP8, int MF>
hipError_t launch_moe_rows(const MoeArgs& a, bool gated, hipStream_t s) {
  const unsigned pairs = a.tokens * a.top_k;
  const unsigned gy = a.by_expert ? a.experts : pairs;
  moe_logits_kernel<E><<<dim3(a.experts, (a.tokens + 3) / 4), 256, 0, s>>>(a);
  moe_route_kernel<<<a.tokens, 64, a.experts * sizeof(double), s>>>(a);
  const dim3 up((unsigned)(((int64_t)a.d_ff + 15) / 16), gy);
  if (gated)
    moe_up_kernel<E, FP8, true, MF><<<up, 512, 0, s>>>(a);
  else
    moe_up_kernel<E, FP8, false, MF><<<up, 512, 0, s>>>(a);
  const dim3 down((unsigned)(((int64_t)a.d_model + 15) / 16), gy);
  moe_down_kernel<E, FP8, MF><<<down, 512, 0, s>>>(a);
  const unsigned blocks = (unsigned)(((int64_t)a.d_model + 255) / 256);
  moe_combine_kernel<E><<<dim3(blocks, a.tokens), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <class E, bool FP8>
hipError_t launch_moe_as(const MoeArgs& a, bool gated, hipStream_t s) {
  if (a.tokens <= 16) return launch_moe_rows<E, FP8, 1>(a, gated, s);
  if (a.tokens <= 32) return launch_moe_rows<E, FP8, 2>(a, gated, s);
  return launch_moe_rows<E, FP8, 4>(a, gated, s);
}

}  // namespace

size_t moe_workspace_bytes(const moe_shape_t& s) { return moe_layout(s).bytes; }

hipError_t launch_moe(const MoeCall& c, int cus, hipStream_t s) {
  (void)cus;
  const moe_shape_t& sh = c.shape;
  const MoeWorkspace l = moe_layout(sh);
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  MoeArgs a{};
  a.tokens = sh.tokens;
  a.d_model = sh.d_model;
  a.d_ff = sh.d_ff;
  a.experts = sh.experts;
  a.top_k = sh.top_k;
  a.act = sh.act;
  a.norm = sh.norm_topk != 0;
  a.by_expert = sh.experts <= sh.tokens * sh.top_k;
  a.X = c.X;
  a.ldx = c.ldx;
  a.R = c.R;
  a.ldr = c.ldr;
  a.W1 = c.W1;
  a.ld1 = c.ld1;
  a.S1 = c.S1;
  a.W2 = c.W2;
  a.ld2 = c.ld2;
  a.S2 = c.S2;
  a.ids = c.ids;
  a.w = c.w;
  a.Y = c.Y;
  a.ldy = c.ldy;
  a.logits = reinterpret_cast<double*>(ws + l.logits);
  a.h_hi = reinterpret_cast<uint16_t*>(ws + l.h);
  a.h_lo = a.h_hi + (size_t)sh.tokens * sh.top_k * l.ldh;
  a.ldh = l.ldh;
  a.part = reinterpret_cast<float*>(ws + l.part);
  const bool fp8 = sh.weight_type == GEMM_TYPE_E4M3, gated = sh.gated != 0;
  if (sh.type == GEMM_TYPE_F16)
    return fp8 ? launch_moe_as<LmF16, true>(a, gated, s) : launch_moe_as<LmF16, false>(a, gated, s);
  return fp8 ? launch_moe_as<LmBF16, true>(a, gated, s) : launch_moe_as<LmBF16, false>(a, gated, s);
}

}  // namespace lasg
