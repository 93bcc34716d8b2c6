// A mixture-of-experts feed-forward layer for a few tokens (at most 64):
//     l[t][e]  = sum_d X[t][d] R[e][d]
//     ids[t]   = the top_k largest l[t], largest first, ties to the lower expert
//     w[t]     = softmax(l[t]) at ids[t], divided by their sum if asked for
//     h[t][s]  = act(W1[e] x) (* the second half of W1's rows when gated), e = ids[t][s]
//     Y[t]     = sum_s w[t][s] W2[e] h[t][s]
//
// What bounds it are the chosen experts' weights, each of which is read once:
// the tokens that chose an expert form the rows of one small product against
// it.  A workgroup takes an expert and 16 NF rows of its weight; its waves take
// equal shares of the columns (consecutive ones: 7 % faster than every eighth
// block of 128), read the weight straight into MFMA operands (16x16x32, the
// tokens as the other operand) and add their fp32 sums in LDS.  Which
// experts there are is known on the device only, so the grids have a row for
// every expert or for every token and slot, whichever is fewer, and workgroups
// whose expert nobody chose, or another row takes, end at once.
//
// Four launches: the logits; the first product, whose workgroups find their
// expert and its tokens from the logits (a token chose an expert if fewer than
// top_k logits come before its own: one comparison per lane and ballot for 64
// experts), beside workgroups that write the choice and its weights down; the
// second product; the sum over a token's slots.  For one token the last two are one.
//
// Measured (us of kernel time; the card reads 6.2 TB/s): 64 tokens, 8 experts of 4096
// x 14336 in bfloat16: 345 (5.5 TB/s) and 196 (5.1); 4 tokens, 64 experts of 4096 x
// 1536 in e4m3: 69 (5.0) and 39 (4.4), logits 4.8, sum 4.7; one token, 8 experts
// of 1024 x 512: 2.4, 6.7 and 4.7, latency throughout.  (Rates from counted bytes.)
//
// The logits are summed in 64 bits: two experts' logits can lie closer than
// fp32 sums of a few thousand terms resolve, and the choice between them is an
// output.  The inner activations h are kept to about 16 (bfloat16) or 22
// (binary16) bits as a pair hi + lo of the 16-bit type, each multiplied by W2:
// rounded to one such number they would cost as much accuracy as the final
// rounding of Y, and the second MFMA is free beside the loads.  In binary16 h
// is clamped to +-65504, the type's range, and the pair cannot hold less than
// 2^-24.  Rows (a token's h for one expert) whose largest |h| is at least kSmallPeak
// lose at most 2^-17 of that by it and are taken as they are.  For the others the
// second product reads h in fp32, which the first writes beside the pair, with the
// largest |h| of every workgroup's columns, and multiplies it by a power of two that brings
// the row's largest to 2^14 .. 2^15: 2^-39 of it is lost.  Such rows take 10 to 20 %
// longer (4 tokens, 64 e4m3 experts: 121 us for 109), the others what the extra
// stores cost, up to half a microsecond in each product.  (Plain stores: one
// atomic maximum per row and workgroup took up to 8 us of the first product.)
// A 16-bit weight may be infinite; lo, of either sign or zero, would then turn an
// infinite sum into NaN, which the sum of hi's products alone settles (high_sum,
// add_low).
#include <type_traits>

#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

namespace {

constexpr int kMaxTokens = 64;   // one wave's lanes hold the tokens
constexpr int kMaxExperts = 1024, kMaxSlots = 32;   // (as lm_capi.cpp allows)
constexpr uint32_t kSmallPeak = 0x3b800000u;   // 2^-8, as the bits of an fp32 number

// Where the parts of the workspace lie (bytes).
struct MoeWorkspace {
  size_t logits, h, part, wide, flags, peaks, bytes;
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
  w.wide = w.part + round256(pairs * s.d_model * sizeof(float));
  const bool narrow = s.type == GEMM_TYPE_F16;
  w.flags = w.wide + (narrow ? round256(pairs * w.ldh * sizeof(float)) : 0);
  w.peaks = w.flags + (narrow ? round256(2 * pairs * sizeof(uint32_t)) : 0);
  w.bytes = w.peaks +
            (narrow ? round256(pairs * (((size_t)s.d_ff + 15) / 16) * sizeof(uint32_t)) : 0);
  return w;
}

struct MoeArgs {
  int tokens, d_model, d_ff, experts, top_k, act;
  bool norm, by_expert;   // by_expert: grid rows are experts, else (token, slot) pairs
  int force_rows;         // rows of a weight per workgroup (host only; 0: by shape)
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
  // Binary16 only: h in fp32 (rows of ldh); for every row whether some |h| is at least
  // kSmallPeak, and whether some workgroup's largest is below it and not zero;
  // the largest |h| (bits) of each of the first product's up_tiles workgroups.
  float* h_wide;
  uint32_t* flags;
  uint32_t* peaks;
  int up_tiles;
  float* part;
};

// Whether a row needs the fp32 values.
__device__ __forceinline__ bool small_row(const MoeArgs& p, int pair) {
  const u32x2 f = *reinterpret_cast<const u32x2*>(p.flags + 2 * pair);
  return f[0] == 0 && f[1] != 0;
}
// The largest |h| (bits) of a row, by one wave, in every lane.
__device__ __forceinline__ uint32_t row_peak(const MoeArgs& p, int pair) {
  uint32_t m = 0;
  for (int b = threadIdx.x % kWave; b < p.up_tiles; b += kWave) {
    const uint32_t x = p.peaks[(int64_t)pair * p.up_tiles + b];
    m = m > x ? m : x;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t x = (uint32_t)__shfl_xor((int)m, d);
    m = m > x ? m : x;
  }
  return m;
}
// The exponent of the power of two that a row is multiplied by (negated: divided by), as a factor.
__device__ __forceinline__ int row_shift(uint32_t peak) {
  const int up = 141 - (int)(peak >> 23);   // 2^14 over the largest's exponent
  return peak == 0 || peak >= kSmallPeak ? 0 : up < 126 ? up : 126;
}
__device__ __forceinline__ float power_of_two(int e) {
  return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}

// h as hi + lo.
template <class E>
__device__ __forceinline__ void split(float h, uint16_t& hi, uint16_t& lo) {
  const bool inf = __builtin_fabsf(h) == __builtin_inff();
  hi = E::bits(h);
  lo = E::bits(inf ? 0.0f : h - E::value(hi));
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// Whether expert o with logit u comes before expert e with logit v: NaN first,
// then larger logits, then lower numbers (a total order whatever the logits).
__device__ __forceinline__ bool before(double u, int o, double v, int e) {
  const bool un = u != u, vn = v != v;
  return un || vn ? un && (!vn || o < e) : u > v || (u == v && o < e);
}

// The tokens that chose `expert`, from the logits, in token order: pair[i] =
// token * top_k + slot.  Returns their number.  Wave w of W looks at the tokens w, w + W,
// ..., four of them at a time.
template <int W>
__device__ __forceinline__ int rows_from_logits(const MoeArgs& p, int expert, int* pair, int* slots) {
  constexpr int BATCH = 4;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
#pragma unroll 1
  for (int t0 = wave; t0 < p.tokens; t0 += W * BATCH) {
    double own[BATCH];
    int place[BATCH] = {};
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (t0 + W * i < p.tokens)
        own[i] = p.logits[(int64_t)(t0 + W * i) * p.experts + expert];
#pragma unroll 1
    for (int o = lane; o < p.experts + lane; o += kWave) {   // (every lane takes part in the ballots)
      double u[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (t0 + W * i < p.tokens)
          u[i] = o < p.experts ? p.logits[(int64_t)(t0 + W * i) * p.experts + o] : 0.0;
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (t0 + W * i < p.tokens)
          place[i] += __popcll(__ballot(o < p.experts && before(u[i], o, own[i], expert)));
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (lane == 0 && t0 + W * i < p.tokens) slots[t0 + W * i] = place[i];
  }
  __syncthreads();
  const bool chose = lane < p.tokens && slots[lane] < p.top_k;
  const uint64_t mask = __ballot(chose);
  if (wave == 0 && chose)
    pair[__popcll(mask & ((uint64_t(1) << lane) - 1))] = lane * p.top_k + slots[lane];
  __syncthreads();
  return __popcll(mask);
}

// The expert in place `slot` of a token's order: lane l holds the logits of the experts
// l, l + 64, ..., and wave w finds the places of the experts w, w + W, ....  At most
// kPairExperts experts.
constexpr int kPairExperts = 256;
template <int W>
__device__ __forceinline__ int expert_from_logits(const MoeArgs& p, int token, int slot, int* found) {
  constexpr int PER_LANE = kPairExperts / kWave;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const double* logits = p.logits + (int64_t)token * p.experts;
  double u[PER_LANE];
#pragma unroll
  for (int c = 0; c < PER_LANE; ++c) {
    const int o = c * kWave + lane;
    u[c] = o < p.experts ? logits[o] : 0.0;
  }
#pragma unroll
  for (int c = 0; c < PER_LANE; ++c) {
    if (c * kWave >= p.experts) break;
#pragma unroll 1
    for (int l = wave; l < kWave && c * kWave + l < p.experts; l += W) {
      const uint64_t bits = __builtin_bit_cast(uint64_t, u[c]);
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)bits, l);
      const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), l);
      const double v = __builtin_bit_cast(double, lo | (uint64_t)hi << 32);
      const int e = c * kWave + l;
      int place = 0;
#pragma unroll
      for (int d = 0; d < PER_LANE; ++d) {
        const int o = d * kWave + lane;
        if (d * kWave < p.experts)
          place += __popcll(__ballot(o < p.experts && before(u[d], o, v, e)));
      }
      if (place == slot && lane == 0) *found = e;
    }
  }
  __syncthreads();
  return *found;
}

// A token's choice and its weights, by one workgroup (beside the product: the
// second product is the first to need them).
template <int W>
__device__ __forceinline__ void route_token(const MoeArgs& p, int t, double* key, double* chosen) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int e = threadIdx.x; e < p.experts; e += 64 * W) key[e] = p.logits[(int64_t)t * p.experts + e];
  __syncthreads();
#pragma unroll 1
  for (int e = wave; e < p.experts; e += W) {
    int place = 0;
#pragma unroll 1
    for (int o = lane; o < p.experts + lane; o += kWave)
      place += __popcll(__ballot(o < p.experts && before(key[o < p.experts ? o : 0], o, key[e], e)));
    if (place < p.top_k && lane == 0) {
      chosen[place] = key[e];
      p.ids[t * p.top_k + place] = e;
    }
  }
  __syncthreads();
  if (wave == 0) {
    // (The first place holds the largest logit.  Divided by the chosen ones' sum,
    // the sum over all experts drops out.)
    const double top = chosen[0];
    const double mine = lane < p.top_k ? exp(chosen[lane] - top) : 0.0;
    double sum = mine;
    if (!p.norm) {
      sum = 0.0;
      for (int e = lane; e < p.experts; e += kWave) sum += exp(key[e] - top);
    }
    sum = wave_sum(sum);
    if (lane < p.top_k) p.w[t * p.top_k + lane] = (float)(mine / sum);
  }
  __syncthreads();
}

// The same from the written choice, for a grid row that stands for an expert, or
// for a (token, slot) pair: then the expert's first pair does the work.
struct Rows {
  int expert, count;   // count == 0: nothing for this workgroup
  bool small;          // NARROW: whether one of them is a small row
};
template <bool NARROW>
__device__ __forceinline__ Rows rows_from_ids(const MoeArgs& p, int grid_row, int* pair) {
  const int lane = threadIdx.x % kWave;
  const int pairs = p.tokens * p.top_k;
  Rows out{p.by_expert ? grid_row : p.ids[grid_row], 0, false};
  for (int q0 = 0; q0 < pairs; q0 += 4 * kWave) {   // (pairs are in token order)
    int id[4];
    bool small[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int q = q0 + u * kWave + lane;
      id[u] = q < pairs ? p.ids[q] : -1;
      small[u] = NARROW && q < pairs ? small_row(p, q) : false;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t mask = __ballot(id[u] == out.expert);
      if (mask == 0) continue;
      if (!p.by_expert && out.count == 0 &&
          q0 + u * kWave + __ffsll((unsigned long long)mask) - 1 != grid_row)
        return Rows{out.expert, 0, false};
      if (threadIdx.x < kWave && id[u] == out.expert)
        pair[out.count + __popcll(mask & ((uint64_t(1) << lane) - 1))] = q0 + u * kWave + lane;
      out.count += __popcll(mask);
      if (NARROW && __ballot(id[u] == out.expert && small[u]) != 0) out.small = true;
    }
  }
  if (out.count > 0) __syncthreads();
  return out;
}

// How a lane reads a block of K columns of 16 rows (128 bytes of each): in two
// chunks of 16 bytes of a weight's row (8 or 16 columns), chunk u of lane group g
// at column chunk(u, g), as the first operands of T MFMAs; MFMA t multiplies eight
// columns of chunk t / PER.
//
// The last, shorter block of a row (Tail): a chunk that crosses the row's end is
// moved back to the row's last columns, and `mask` keeps those of them that no
// other chunk covers, in weight and tokens alike (a masked infinity must not
// meet a zero).  Rows shorter than a chunk are gathered by element.
template <class E, bool FP8>
struct Block {
  static constexpr int K = FP8 ? 128 : 64, COLS = FP8 ? 16 : 8, T = K / 32, PER = T / 2;
  typedef typename E::vec8 vec8;
  static __device__ __forceinline__ int chunk(int u, int g) { return K / 2 * u + COLS * g; }

  struct Tail {
    int at[2];        // first column
    u32x4 mask[T];    // of the eight columns of MFMA t, 16 bits each
    u32x4 mask8[2];   // e4m3: of the chunk's 16 bytes
    int tiny;         // the row's columns, if fewer than a chunk (else 0)
    __device__ __forceinline__ Tail(int k0, int cols, int g) {
      tiny = cols < COLS ? cols : 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int first = k0 + chunk(u, g);
        at[u] = tiny ? 0 : first < cols - COLS ? first : cols - COLS;
        // Columns at[u] + c count if they are not before `first` (nor past the end).
        const int from = first - at[u], to = tiny ? (first == 0 ? cols : 0) : COLS;
#pragma unroll
        for (int x = 0; x < PER; ++x)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int c = 8 * x + 2 * d;
            mask[u * PER + x][d] = (c >= from && c < to ? 0xffffu : 0u) |
                                   (c + 1 >= from && c + 1 < to ? 0xffff0000u : 0u);
          }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m |= 4 * d + e >= from && 4 * d + e < to ? 0xffu << (8 * e) : 0u;
          mask8[u][d] = m;
        }
      }
    }
  };

  u32x4 c[2];   // as loaded (widened only when it is multiplied: a block on its way takes 8 registers)
  __device__ __forceinline__ vec8 operand(int t) const {
    if constexpr (FP8)
      return t % 2 ? E::widen(c[t / 2][2], c[t / 2][3]) : E::widen(c[t / 2][0], c[t / 2][1]);
    else
      return __builtin_bit_cast(vec8, c[t]);
  }
  __device__ __forceinline__ void load(const uint8_t* row, int k0, int g) {
#pragma unroll
    for (int u = 0; u < 2; ++u) c[u] = load16(row + (k0 + chunk(u, g)) * (FP8 ? 1 : 2));
  }
  __device__ __forceinline__ void load(const uint8_t* row, const Tail& tail) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x4 x = tail.tiny ? gather(row, tail.tiny * (FP8 ? 1 : 2))
                                : load16(row + tail.at[u] * (FP8 ? 1 : 2));
      c[u] = x & (FP8 ? tail.mask8[u] : tail.mask[u * PER]);
    }
  }
  static __device__ __forceinline__ vec8 tokens(const uint16_t* row, int k0, int g, int t) {
    return __builtin_bit_cast(vec8, load16(row + k0 + chunk(t / PER, g) + 8 * (t % PER)));
  }
  static __device__ __forceinline__ vec8 tokens(const uint16_t* row, const Tail& tail, int t) {
    const int at = tail.at[t / PER] + 8 * (t % PER);
    const u32x4 x = tail.tiny ? gather(reinterpret_cast<const uint8_t*>(row + at), 2 * (tail.tiny - at))
                              : load16(row + at);
    return __builtin_bit_cast(vec8, x & tail.mask[t]);
  }
  // Eight fp32 values times `factor` as two numbers of the type.
  static __device__ __forceinline__ void split8(const float* at, float factor, vec8& hi, vec8& lo) {
    const f32x4 x[2] = {*reinterpret_cast<const f32x4_any*>(at),
                        *reinterpret_cast<const f32x4_any*>(at + 4)};
    uint16_t h[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split<E>(x[e / 4][e % 4] * factor, h[e], l[e]);
    hi = __builtin_bit_cast(vec8, h);
    lo = __builtin_bit_cast(vec8, l);
  }
  // The tokens from a row of h_wide.  (Its rows are padded to 128 columns, so what a tail's
  // mask takes away may be read.)
  static __device__ __forceinline__ void tokens(const float* row, float factor, int k0, int g, int t,
                                                vec8& hi, vec8& lo) {
    split8(row + k0 + chunk(t / PER, g) + 8 * (t % PER), factor, hi, lo);
  }
  static __device__ __forceinline__ void tokens(const float* row, float factor, const Tail& tail,
                                                int t, vec8& hi, vec8& lo) {
    split8(row + tail.at[t / PER] + 8 * (t % PER), factor, hi, lo);
    hi = __builtin_bit_cast(vec8, __builtin_bit_cast(u32x4, hi) & tail.mask[t]);
    lo = __builtin_bit_cast(vec8, __builtin_bit_cast(u32x4, lo) & tail.mask[t]);
  }
  // The first `bytes` (fewer than 32) bytes of a row, up to 16.
  static __device__ __forceinline__ u32x4 gather(const uint8_t* row, int bytes) {
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int e = 0; e < 16 && e < bytes; ++e) {
      const uint64_t b = (uint64_t)row[e] << (8 * (e % 8));
      lo |= e < 8 ? b : 0;
      hi |= e < 8 ? 0 : b;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
};

}  // namespace

// Logits of one expert and TT tokens per workgroup, its four waves splitting
// the columns; products and sums in 64 bits.
template <class E, int TT>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeArgs p) {
  __shared__ double sums[4][TT];
  const int e = blockIdx.x, t0 = TT * blockIdx.y;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  if (E::kNarrow && blockIdx.x == 0 && blockIdx.y == 0)
    for (int q = threadIdx.x; q < 2 * p.tokens * p.top_k; q += 256) p.flags[q] = 0;
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

// Adds the W waves' sums `total` of F fragments in LDS, in a fixed order (the
// upper half of the waves first put theirs there, the lower half add their
// own, so that half the space serves) and leaves them in part, still to be added up by joined().
template <int F, int H>
__device__ __forceinline__ void join(const f32x4 (&total)[F], float (&part)[H][F][256], int wave,
                                     int lane) {
  if (wave >= H) {
#pragma unroll
    for (int f = 0; f < F; ++f) *reinterpret_cast<f32x4*>(&part[wave - H][f][4 * lane]) = total[f];
  }
  __syncthreads();
  if (wave < H) {
#pragma unroll
    for (int f = 0; f < F; ++f)
      *reinterpret_cast<f32x4*>(&part[wave][f][4 * lane]) += total[f];
  }
  __syncthreads();
}
template <int F, int H>
__device__ __forceinline__ float joined(const float (&part)[H][F][256], int f, int at) {
  if constexpr (H == 2) return part[0][f][at] + part[1][f][at];
  return (part[0][f][at] + part[1][f][at]) + (part[2 % H][f][at] + part[3 % H][f][at]);
}

// Waves of a workgroup of the two products.  With many tokens a wave's sums fill
// the registers of half a SIMD; workgroups of four waves then leave room for
// two on a compute unit, one starting or ending while the other reads.
constexpr int waves_of(int mf) { return mf == 4 ? 4 : 8; }

// A wave's whole blocks first .. end - 1 of F weight rows' fragments: the next
// block of weights is on its way while this one is multiplied.  The tokens of a
// block are asked for before the next weights (loads return in order), all at
// once where they fit the registers.  `load_weights(B (&)[F], kb)`,
// `load_tokens(X&, i, kb)`, `multiply(B (&)[F], X&, i, kb)`; `count` tokens of at
// most 16 MF.  AHEAD false: without the block ahead, which pays with 16-bit
// weights (64 tokens, 8 experts: 405 -> 344 and 234 -> 198 us); e4m3 blocks hold twice
// the columns, and the registers are worth more as occupancy (4 tokens, 64
// experts: 73 and 49 us without, 100 and 65 with).
template <int MF, int F, int ALL, bool AHEAD, class B, class X, class LW, class LT, class M>
__device__ __forceinline__ void stream_blocks(int first, int end, int count, LW load_weights,
                                              LT load_tokens, M multiply) {
  if (first >= end) return;
  auto run = [&](auto active) __attribute__((always_inline)) {
    constexpr int MA = decltype(active)::value, HELD = MA < ALL ? MA : ALL;
    B weights[AHEAD ? 2 : 1][F];
    if constexpr (AHEAD) load_weights(weights[0], first);
    for (int kb = first; kb < end; kb += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = kb + u;
        if (at >= end) break;
        X tokens[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) load_tokens(tokens[i], i, at);
        if constexpr (AHEAD)
          load_weights(weights[1 - u], at + 1 < end ? at + 1 : at);
        else
          load_weights(weights[0], at);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MA; ++i) {
          if (i >= HELD) load_tokens(tokens[i % HELD], i, at);
          multiply(weights[AHEAD ? u : 0], tokens[i % HELD], i, at);
        }
      }
    }
  };
  if (count <= 16 || MF == 1)
    run(std::integral_constant<int, 1>());
  else if (count <= 32 || MF == 2)
    run(std::integral_constant<int, MF < 2 ? MF : 2>());
  else
    run(std::integral_constant<int, MF>());
}

// Sums of the products of hi and of lo as one.
__device__ __forceinline__ f32x4 add_low(f32x4 hi, f32x4 lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    hi[e] = __builtin_fabsf(hi[e]) < __builtin_inff() ? hi[e] + lo[e] : hi[e];
  return hi;
}

// The sum of hi's products by one lane, for an element that came out NaN (sums
// of their own in the loop, as one token's, would not fit the registers of wide tiles).
// A NaN among the values ends it at once; only an infinite weight reads the row.
// In binary16 it is the sum of h itself, whose hi may be zero where h is not.
template <class E>
__device__ __forceinline__ float high_sum(const uint16_t* w, const float* h, int n) {
  float s = 0.0f;
#pragma unroll 1
  for (int k = 0; k < n && s == s; ++k) s = __builtin_fmaf(E::value(w[k]), h[k], s);
  return s;
}
template <class E>
__device__ __forceinline__ float high_sum(const uint16_t* w, const uint16_t* hi, int n) {
  float s = 0.0f;
#pragma unroll 1
  for (int k = 0; k < n && s == s; k += 8) {
    const u32x4 a = load8h_upto(w + k, n - k), b = load8h_upto(hi + k, n - k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      s = __builtin_fmaf(E::value((uint16_t)(a[i / 2] >> (16 * (i % 2)))),
                         E::value((uint16_t)(b[i / 2] >> (16 * (i % 2)))), s);
  }
  return s;
}

// h for 16 NF inner columns of one expert and all its tokens (at most 16 MF).
template <class E, bool FP8, bool GATED, int MF, int NF>
__global__ void __launch_bounds__(64 * waves_of(MF))
__attribute__((amdgpu_waves_per_eu(MF == 1 ? 4 : 2))) moe_up_kernel(MoeArgs p) {
  constexpr int SIDES = GATED ? 2 : 1, W = waves_of(MF);
  __shared__ __attribute__((aligned(16))) float part[W / 2][SIDES * NF * MF][256];
  __shared__ int pair[kMaxTokens], slots[kMaxTokens], found;
  __shared__ double key[kMaxExperts], chosen[kMaxSlots];
  __shared__ uint32_t peak[E::kNarrow ? kMaxTokens : 1];
  if (blockIdx.y == gridDim.y - 1) {   // (one grid row past the experts: the tokens' choices)
    for (int t = blockIdx.x; t < p.tokens; t += gridDim.x) route_token<W>(p, t, key, chosen);
    return;
  }
  const int expert = p.by_expert ? blockIdx.y
                                 : expert_from_logits<W>(p, blockIdx.y / p.top_k,
                                                      blockIdx.y % p.top_k, &found);
  int count = 1;
  if (p.tokens == 1 && !p.by_expert) {
    if (threadIdx.x == 0) pair[0] = blockIdx.y;
    __syncthreads();
  } else {
    count = rows_from_logits<W>(p, expert, pair, slots);
  }
  // (By pair, an expert's first pair does the work.)
  if (count == 0 || (!p.by_expert && pair[0] != (int)blockIdx.y)) return;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, g = lane / 16;
  const int n0 = 16 * NF * blockIdx.x;
  const int D = p.d_model, I = p.d_ff;
  const int64_t rows1 = (int64_t)SIDES * I;
  const uint16_t* x[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int at = 16 * i + r < count ? 16 * i + r : count - 1;
    x[i] = p.X + (int64_t)(pair[at] / p.top_k) * p.ldx;
  }
  const uint8_t* w[SIDES][NF];
  const int64_t rbs = (rows1 + 127) / 128;
  const int kbs = (D + 127) / 128;
  // Scales of a fragment's rows: the second half of W1 may start inside a block
  // of 128 rows, so a fragment may lie in two; `edge` is its first row (of 16) in the second.
  const float* scale[SIDES][NF];
  int edge[SIDES][NF];
#pragma unroll
  for (int side = 0; side < SIDES; ++side)
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int n = n0 + 16 * j + r < I ? n0 + 16 * j + r : I - 1;   // (rows past the end: never stored)
      w[side][j] = static_cast<const uint8_t*>(p.W1) +
                   ((int64_t)expert * rows1 + (int64_t)side * I + n) * p.ld1 * (FP8 ? 1 : 2);
      if constexpr (FP8) {
        int64_t first = (int64_t)side * I + n0 + 16 * j;
        if (first >= rows1) first = rows1 - 1;
        scale[side][j] = p.S1 + (int64_t)expert * kbs * rbs + first / 128;
        edge[side][j] = first / 128 + 1 < rbs ? 128 - (int)(first % 128) : 16;
      }
    }
  f32x4 total[SIDES * NF * MF];
#pragma unroll
  for (int f = 0; f < SIDES * NF * MF; ++f) total[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  typedef Block<E, FP8> B;
  constexpr int F = SIDES * NF;
  struct X {
    typename E::vec8 v[B::T];
    float s0[FP8 ? F : 1], s1[FP8 ? F : 1];   // scales of the block (with the first 16 tokens)
  };
  auto load_scales = [&](X& t, int kb) __attribute__((always_inline)) {
    if constexpr (FP8) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const float* s = scale[f / NF][f % NF] + kb * rbs;
        t.s0[f] = uniform_value(s);
        t.s1[f] = uniform_value(s + (edge[f / NF][f % NF] < 16 ? 1 : 0));
      }
    }
  };
  auto multiply = [&](B (&wb)[F], X& t, int i, int) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      f32x4& sum = total[f * MF + i];
      f32x4 v = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum;
#pragma unroll
      for (int m = 0; m < B::T; ++m) v = E::mfma(wb[f].operand(m), t.v[m], v);
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum[e] = __builtin_fmaf(v[e], 4 * g + e < edge[f / NF][f % NF] ? t.s0[f] : t.s1[f], sum[e]);
      } else {
        sum = v;
      }
    }
  };
  const int full = D / B::K;
  stream_blocks<MF, F, FP8 ? 1 : 4, !FP8, B, X>(
      full * wave / W, full * (wave + 1) / W, count,
      [&](B (&wb)[F], int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < F; ++f) wb[f].load(w[f / NF][f % NF], kb * B::K, g);
      },
      [&](X& t, int i, int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < B::T; ++m) t.v[m] = B::tokens(x[i], kb * B::K, g, m);
        load_scales(t, kb);
      },
      multiply);
  if (full * B::K < D && wave == W - 1) {
    const typename B::Tail tail(full * B::K, D, g);
    B wb[F];
#pragma unroll
    for (int f = 0; f < F; ++f) wb[f].load(w[f / NF][f % NF], tail);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if (16 * i >= count) break;
      X t;
#pragma unroll
      for (int m = 0; m < B::T; ++m) t.v[m] = B::tokens(x[i], tail, m);
      load_scales(t, full);
      multiply(wb, t, i, full);
    }
  }
  if (E::kNarrow && threadIdx.x < kMaxTokens) peak[threadIdx.x] = 0;
  join(total, part, wave, lane);
  for (int v = threadIdx.x; v < NF * MF * 256; v += 64 * W) {
    const int f = v / 256, at = v % 256;
    const int token = 16 * (f % MF) + (at / 4) % 16;
    const int n = n0 + 16 * (f / MF) + 4 * (at / 64) + at % 4;
    if (token >= count || n >= I) continue;
    float s[SIDES];
#pragma unroll
    for (int side = 0; side < SIDES; ++side) {
      const int q = side * NF * MF + f;
      s[side] = joined(part, q, at);
    }
    float h = apply_act(s[0], p.act);
    if constexpr (GATED) h *= s[SIDES - 1];
    const bool inf = __builtin_fabsf(h) == __builtin_inff();   // (infinities and NaN stay)
    if (!inf) h = h > E::kMax ? E::kMax : h < -E::kMax ? -E::kMax : h;
    const int64_t at_h = (int64_t)pair[token] * p.ldh + n;
    split<E>(h, p.h_hi[at_h], p.h_lo[at_h]);
    if constexpr (E::kNarrow) {
      p.h_wide[at_h] = h;
      atomicMax(&peak[token], __builtin_bit_cast(uint32_t, h) & 0x7fffffffu);
    }
  }
  if constexpr (E::kNarrow) {
    __syncthreads();
    if ((int)threadIdx.x < count) {
      const int q = pair[threadIdx.x];
      const uint32_t m = peak[threadIdx.x];
      p.peaks[(int64_t)q * gridDim.x + blockIdx.x] = m;
      if (m >= kSmallPeak)
        p.flags[2 * q] = 1;
      else if (m != 0)
        p.flags[2 * q + 1] = 1;
    }
  }
}

// h W2 of 16 NF output columns of one expert and all its tokens, per pair.
template <class E, bool FP8, int MF, int NF>
__global__ void __launch_bounds__(64 * waves_of(MF))
__attribute__((amdgpu_waves_per_eu(MF == 1 ? 4 : 2))) moe_down_kernel(MoeArgs p) {
  constexpr int W = waves_of(MF);
  __shared__ __attribute__((aligned(16))) float part[W / 2][NF * MF][256];
  __shared__ int pair[kMaxTokens], shift[E::kNarrow ? kMaxTokens : 1];
  const Rows rows = rows_from_ids<E::kNarrow>(p, blockIdx.y, pair);
  if (rows.count == 0) return;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, g = lane / 16;
  const int n0 = 16 * NF * blockIdx.x;
  const int D = p.d_model, I = p.d_ff;
  int64_t h_row[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int at = 16 * i + r < rows.count ? 16 * i + r : rows.count - 1;
    h_row[i] = pair[at] * p.ldh;
  }
  const uint8_t* w[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int n = n0 + 16 * j + r < D ? n0 + 16 * j + r : D - 1;
    w[j] = static_cast<const uint8_t*>(p.W2) +
           ((int64_t)rows.expert * D + n) * p.ld2 * (FP8 ? 1 : 2);
  }
  const int64_t rbs = (D + 127) / 128;
  const int kbs = (I + 127) / 128;
  // (16 NF divides 128: one scale for all the rows)
  const float* scale = FP8 ? p.S2 + rows.expert * kbs * rbs + n0 / 128 : nullptr;
  f32x4 total[NF * MF];
#pragma unroll
  for (int f = 0; f < NF * MF; ++f) total[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  typedef Block<E, FP8> B;
  struct X {
    typename E::vec8 hi[B::T], lo[B::T];
    float scale;
  };
  auto multiply = [&](B (&wb)[NF], X& t, int i, int) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      f32x4& sum = total[j * MF + i];
      f32x4 v = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum;
#pragma unroll
      for (int m = 0; m < B::T; ++m) {
        const typename E::vec8 a = wb[j].operand(m);
        v = E::mfma(a, t.lo[m], v);
        v = E::mfma(a, t.hi[m], v);
      }
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(v[e], t.scale, sum[e]);
      } else {
        sum = v;
      }
    }
  };
  const int full = I / B::K;
  auto load_weights = [&](B (&wb)[NF], int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NF; ++j) wb[j].load(w[j], kb * B::K, g);
  };
  auto block_scale = [&](int kb) __attribute__((always_inline)) {
    return FP8 ? uniform_value(scale + kb * rbs) : 1.0f;
  };
  const int first = full * wave / W, end = full * (wave + 1) / W;
  const bool small = E::kNarrow && rows.small;
  float factor[E::kNarrow ? MF : 1];
  if (!small) {
    stream_blocks<MF, NF, FP8 ? 1 : 2, !FP8, B, X>(
        first, end, rows.count, load_weights,
        [&](X& t, int i, int kb) __attribute__((always_inline)) {
#pragma unroll
          for (int m = 0; m < B::T; ++m) {
            t.hi[m] = B::tokens(p.h_hi + h_row[i], kb * B::K, g, m);
            t.lo[m] = B::tokens(p.h_lo + h_row[i], kb * B::K, g, m);
          }
          t.scale = block_scale(kb);
        },
        multiply);
  } else if constexpr (E::kNarrow) {
    // h in fp32, for a workgroup with a small row: a block at a time, the values of one
    // MFMA after the other (all of a block's would not fit the registers).  The products
    // of the other rows are added in the same order and give the same bits.
    for (int t = wave; t < rows.count; t += W) {
      const int s = row_shift(row_peak(p, pair[t]));
      if (lane == 0) shift[t] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MF; ++i)
      factor[i] = power_of_two(shift[16 * i + r < rows.count ? 16 * i + r : rows.count - 1]);
#pragma unroll 1
    for (int kb = first; kb < end; ++kb) {
      B wb[NF];
      load_weights(wb, kb);
      const float s = block_scale(kb);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        if (16 * i >= rows.count) break;
        f32x4 v[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j)
          v[j] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : total[j * MF + i];
#pragma unroll
        for (int m = 0; m < B::T; ++m) {
          typename E::vec8 hi, lo;
          B::tokens(p.h_wide + h_row[i], factor[i], kb * B::K, g, m, hi, lo);
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const typename E::vec8 a = wb[j].operand(m);
            v[j] = E::mfma(a, lo, v[j]);
            v[j] = E::mfma(a, hi, v[j]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          f32x4& sum = total[j * MF + i];
          if constexpr (FP8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(v[j][e], s, sum[e]);
          } else {
            sum = v[j];
          }
        }
      }
    }
  }
  if (full * B::K < I && wave == W - 1) {
    const typename B::Tail tail(full * B::K, I, g);
    B wb[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) wb[j].load(w[j], tail);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if (16 * i >= rows.count) break;
      X t;
#pragma unroll
      for (int m = 0; m < B::T; ++m) {
        if (!small) {
          t.hi[m] = B::tokens(p.h_hi + h_row[i], tail, m);
          t.lo[m] = B::tokens(p.h_lo + h_row[i], tail, m);
        } else if constexpr (E::kNarrow) {
          B::tokens(p.h_wide + h_row[i], factor[i], tail, m, t.hi[m], t.lo[m]);
        }
      }
      t.scale = block_scale(full);
      multiply(wb, t, i, full);
    }
  }
  join(total, part, wave, lane);
  for (int v = threadIdx.x; v < NF * MF * 256; v += 64 * W) {
    const int f = v / 256, at = v % 256;
    const int token = 16 * (f % MF) + (at / 4) % 16;
    const int col = n0 + 16 * (f / MF) + 4 * (at / 64) + at % 4;
    if (token >= rows.count || col >= D) continue;
    float y = joined(part, f, at);
    if (small) y *= power_of_two(-shift[E::kNarrow ? token : 0]);
    if constexpr (!FP8) {
      const int64_t h_at = (int64_t)pair[token] * p.ldh;
      const uint16_t* w_at =
          static_cast<const uint16_t*>(p.W2) + ((int64_t)rows.expert * D + col) * p.ld2;
      if (y != y) {
        if constexpr (E::kNarrow)
          y = high_sum<E>(w_at, p.h_wide + h_at, I);
        else
          y = high_sum<E>(w_at, p.h_hi + h_at, I);
      }
    }
    p.part[(int64_t)pair[token] * D + col] = y;
  }
}

// A token's slots added in their order (no atomics: the same bits every time).
template <class E>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeArgs p) {
  const int t = blockIdx.y, d = blockIdx.x * 256 + threadIdx.x;
  if (d >= p.d_model) return;
  const float* part = p.part + (int64_t)t * p.top_k * p.d_model + d;
  const float* w = p.w + t * p.top_k;
  float s = 0.0f;
#pragma unroll 8
  for (int q = 0; q < p.top_k; ++q) s = __builtin_fmaf(w[q], part[(int64_t)q * p.d_model], s);
  p.Y[t * p.ldy + d] = E::bits(s);
}

// One token: 16 columns of Y per workgroup from all its experts.  The units of
// work are (slot, block of columns), wave w taking an eighth of them.  The order of the
// sum is fixed by the shape.
template <class E, bool FP8>
__global__ void __launch_bounds__(512) moe_down_token_kernel(MoeArgs p) {
  __shared__ __attribute__((aligned(16))) float part[4][1][256];
  typedef Block<E, FP8> B;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, g = lane / 16;
  const int n0 = 16 * blockIdx.x;
  const int D = p.d_model, I = p.d_ff;
  const int n = n0 + r < D ? n0 + r : D - 1;
  const int64_t rbs = (D + 127) / 128;
  const int kbs = (I + 127) / 128, full = I / B::K;
  const int mine = p.ids[lane < p.top_k ? lane : 0];
  float weight = p.w[lane < p.top_k ? lane : 0];
  const bool small = E::kNarrow && small_row(p, lane < p.top_k ? lane : 0);
  f32x4 total[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
  auto row = [&](int s) __attribute__((always_inline)) {
    const int expert = __builtin_amdgcn_readlane(mine, s);
    return static_cast<const uint8_t*>(p.W2) + ((int64_t)expert * D + n) * p.ld2 * (FP8 ? 1 : 2);
  };
  auto add = [&](f32x4 v, int s, int kb) __attribute__((always_inline)) {
    float f = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), s));
    if constexpr (FP8)
      f *= p.S2[__builtin_amdgcn_readlane(mine, s) * kbs * rbs + kb * rbs + n0 / 128];
#pragma unroll
    for (int e = 0; e < 4; ++e) total[0][e] = __builtin_fmaf(v[e], f, total[0][e]);
  };
  auto product = [&](const B& wb, const typename E::vec8 (&hi)[B::T],
                     const typename E::vec8 (&lo)[B::T]) __attribute__((always_inline)) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f}, rest = v;
#pragma unroll
    for (int t = 0; t < B::T; ++t) {
      v = E::mfma(wb.operand(t), hi[t], v);
      rest = E::mfma(wb.operand(t), lo[t], rest);
    }
    return FP8 ? v + rest : add_low(v, rest);
  };
  const int units = p.top_k * full, end = units * (wave + 1) / 8;
  // SMALL: some slot's row is small, h is taken in fp32 (a unit at a time).
  auto products = [&](auto is_small) __attribute__((always_inline)) {
    constexpr bool SMALL = decltype(is_small)::value;
    constexpr int AHEAD = SMALL ? 1 : FP8 ? 2 : 4;   // units whose loads are in flight together
    int shift = 0;   // lane s: of slot s
    if constexpr (SMALL) {
      for (int s = 0; s < p.top_k; ++s) {
        const int x = row_shift(row_peak(p, s));
        if (lane == s) shift = x;
      }
      weight *= power_of_two(-shift);
    }
    auto factor = [&](int s) __attribute__((always_inline)) {
      return power_of_two(__builtin_amdgcn_readlane(shift, s));
    };
    for (int u0 = units * wave / 8; u0 < end; u0 += AHEAD) {
      B wb[AHEAD];
      typename E::vec8 hi[AHEAD][B::T], lo[AHEAD][B::T];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int u = u0 + a < end ? u0 + a : end - 1;
        const int s = u / full, kb = u % full;
        wb[a].load(row(s), kb * B::K, g);
#pragma unroll
        for (int t = 0; t < B::T; ++t) {
          if constexpr (SMALL) {
            B::tokens(p.h_wide + s * p.ldh, factor(s), kb * B::K, g, t, hi[a][t], lo[a][t]);
          } else {
            hi[a][t] = B::tokens(p.h_hi + s * p.ldh, kb * B::K, g, t);
            lo[a][t] = B::tokens(p.h_lo + s * p.ldh, kb * B::K, g, t);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // (all issued before anything waits)
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        if (u0 + a >= end) break;
        add(product(wb[a], hi[a], lo[a]), (u0 + a) / full, (u0 + a) % full);
      }
    }
    if (full * B::K < I) {
      const typename B::Tail tail(full * B::K, I, g);
#pragma unroll 1
      for (int s = wave; s < p.top_k; s += 8) {
        B wb;
        wb.load(row(s), tail);
        typename E::vec8 hi[B::T], lo[B::T];
#pragma unroll
        for (int t = 0; t < B::T; ++t) {
          if constexpr (SMALL) {
            B::tokens(p.h_wide + s * p.ldh, factor(s), tail, t, hi[t], lo[t]);
          } else {
            hi[t] = B::tokens(p.h_hi + s * p.ldh, tail, t);
            lo[t] = B::tokens(p.h_lo + s * p.ldh, tail, t);
          }
        }
        add(product(wb, hi, lo), s, full);
      }
    }
  };
  if constexpr (E::kNarrow) {
    if (__ballot(small) != 0)
      products(std::true_type());
    else
      products(std::false_type());
  } else {
    products(std::false_type());
  }
  join(total, part, wave, lane);
  if (threadIdx.x < 16 && n0 + (int)threadIdx.x < D) {
    const int at = 64 * (threadIdx.x / 4) + threadIdx.x % 4;   // (column 0 of the result: the token)
    float y = joined(part, 0, at);
    if constexpr (E::kNarrow && !FP8) {
      if (y != y) {   // (an infinite weight may have met an hi of zero: see high_sum)
        y = 0.0f;
        for (int s = 0; s < p.top_k; ++s) {
          const uint16_t* w_at = static_cast<const uint16_t*>(p.W2) +
                                 ((int64_t)p.ids[s] * D + n0 + threadIdx.x) * p.ld2;
          y = __builtin_fmaf(p.w[s], high_sum<E>(w_at, p.h_wide + s * p.ldh, I), y);
        }
      }
    }
    p.Y[n0 + threadIdx.x] = E::bits(y);
  }
}

namespace {

// Tiles of 16 NF rows: the widest that leaves two workgroups per compute unit
// (tokens are read once per workgroup, and its start and end cost a few microseconds).
int row_tiles(int64_t n, int64_t grid_rows, int widest, int cus, int force_rows) {
  if (force_rows != 0) return force_rows / 16 < widest ? force_rows / 16 : widest;
  int nf = widest;
  while (nf > 1 && (n + 16 * nf - 1) / (16 * nf) * grid_rows < 2 * cus) nf /= 2;
  return nf;
}

template <class E, bool FP8, int MF>
hipError_t launch_moe_rows(MoeArgs a, bool gated, int cus, hipStream_t s) {
  const int pairs = a.tokens * a.top_k;
  const int rows = a.experts < pairs ? a.experts : pairs;   // experts at work, at most
  if (a.tokens == 1)
    moe_logits_kernel<E, 1><<<a.experts, 256, 0, s>>>(a);
  else if (a.tokens == 2)
    moe_logits_kernel<E, 2><<<a.experts, 256, 0, s>>>(a);
  else
    moe_logits_kernel<E, 4><<<dim3(a.experts, (a.tokens + 3) / 4), 256, 0, s>>>(a);
  const int up_rows = a.by_expert ? a.experts : pairs;
  const int first_rows = up_rows + 1;   // (and one for the tokens' choices)
  const auto grid = [](int n, int nf, int y) {
    return dim3((unsigned)(((int64_t)n + 16 * nf - 1) / (16 * nf)), y);
  };
  // (With e4m3 weights and 64 tokens the widest tile does not fit the registers.)
  constexpr int WIDE = FP8 && MF == 4 ? 2 : 4;
  const int up = row_tiles(a.d_ff, rows, gated ? WIDE / 2 : WIDE, cus, a.force_rows);
  const auto launch_up = [&](auto is_gated, auto nf) {
    constexpr int NF = decltype(nf)::value;
    a.up_tiles = (int)grid(a.d_ff, NF, 1).x;
    moe_up_kernel<E, FP8, decltype(is_gated)::value, MF, NF>
        <<<grid(a.d_ff, NF, first_rows), 64 * waves_of(MF), 0, s>>>(a);
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, WIDE> wide{};
  constexpr std::integral_constant<int, WIDE / 2> half{};
  if (gated)
    up == WIDE / 2 ? launch_up(std::true_type(), half) : launch_up(std::true_type(), one);
  else
    up == WIDE ? launch_up(std::false_type(), wide)
    : up == 2  ? launch_up(std::false_type(), two)
               : launch_up(std::false_type(), one);
  // (One token: 16 columns of Y from all its experts per workgroup.)
  if (a.tokens == 1) {
    moe_down_token_kernel<E, FP8><<<grid(a.d_model, 1, 1), 512, 0, s>>>(a);
    return hipGetLastError();
  }
  const int down = row_tiles(a.d_model, rows, 4, cus, a.force_rows);
  if (down == 4)
    moe_down_kernel<E, FP8, MF, 4><<<grid(a.d_model, 4, up_rows), 64 * waves_of(MF), 0, s>>>(a);
  else if (down == 2)
    moe_down_kernel<E, FP8, MF, 2><<<grid(a.d_model, 2, up_rows), 64 * waves_of(MF), 0, s>>>(a);
  else
    moe_down_kernel<E, FP8, MF, 1><<<grid(a.d_model, 1, up_rows), 64 * waves_of(MF), 0, s>>>(a);
  const unsigned blocks = (unsigned)(((int64_t)a.d_model + 255) / 256);
  moe_combine_kernel<E><<<dim3(blocks, a.tokens), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <class E, bool FP8>
hipError_t launch_moe_as(const MoeArgs& a, bool gated, int cus, hipStream_t s) {
  if (a.tokens <= 16) return launch_moe_rows<E, FP8, 1>(a, gated, cus, s);
  if (a.tokens <= 32) return launch_moe_rows<E, FP8, 2>(a, gated, cus, s);
  return launch_moe_rows<E, FP8, 4>(a, gated, cus, s);
}

}  // namespace

size_t moe_workspace_bytes(const moe_shape_t& s) { return moe_layout(s).bytes; }

hipError_t launch_moe(const MoeCall& c, int cus, int force_rows, hipStream_t s) {
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
  a.by_expert = sh.experts <= sh.tokens * sh.top_k || sh.experts > kPairExperts;
  a.force_rows = force_rows;
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
  if (sh.type == GEMM_TYPE_F16) {
    a.h_wide = reinterpret_cast<float*>(ws + l.wide);
    a.flags = reinterpret_cast<uint32_t*>(ws + l.flags);
    a.peaks = reinterpret_cast<uint32_t*>(ws + l.peaks);
  }
  const bool fp8 = sh.weight_type == GEMM_TYPE_E4M3, gated = sh.gated != 0;
  if (sh.type == GEMM_TYPE_F16)
    return fp8 ? launch_moe_as<LmF16, true>(a, gated, cus, s)
               : launch_moe_as<LmF16, false>(a, gated, cus, s);
  return fp8 ? launch_moe_as<LmBF16, true>(a, gated, cus, s)
             : launch_moe_as<LmBF16, false>(a, gated, cus, s);
}

}  // namespace lasg
