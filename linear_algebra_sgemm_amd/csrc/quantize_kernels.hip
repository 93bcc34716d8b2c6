// Block quantisation to e4m3: of every block of 128 columns of a row (or of
// every 128 x 128 block) the scale s = max(amax / 448, 2^-126) and the values
// x / s rounded to e4m3 (to nearest, ties to even), for the matrix as it lies,
// for its transpose, or for both from one read.
//
// 448 is e4m3's largest value, so no quotient rounds past it and nothing has to
// saturate.  Magnitudes are compared as the integers of their bits without the
// sign, an order in which NaN is above infinity: a NaN makes its block's scale
// and all its values NaN, an infinity makes the scale infinite (finite values of
// the block become 0 and the infinities NaN), as the formula says.  The lower bound on s
// keeps 1 / s finite; a block of zeros has s = 2^-126 and values 0.
//
// The quotient comes from the block's correctly rounded reciprocal r: q0 = x r,
// then q = q0 - r (q0 s - x) with fused multiply-adds, which is x / s correctly
// rounded (Markstein's theorem) unless the remainder underflows.  Three operations instead
// of a division's ten.  (The remainder with this sign leaves -0 as it is; x - q0 s,
// added, gave +0.)  Quotients that e4m3 does not round to 0 are above 2^-10, their
// remainders multiples of 2^-57 s: representable for s >= 2^-60.  Only bfloat16 has smaller
// blocks of 16-bit values; there x and s are first multiplied by 2^64, exactly.
// For 16-bit inputs scale and quotient are fp32 numbers.  For fp32 inputs
// they are formed in 64 bits and rounded once: rounded twice, one or two of 4096 x
// 4096 weights went to the wrong side of the middle between two e4m3 numbers.  And
// they are the exact quotient's: 448 x / amax with neither factor rounded, since
// values of few bits (16-bit ones held in fp32) meet such middles, and a rounded
// amax / 448 sent 210 of 280000 pairs of them to the odd neighbour.
// The 64-bit quotient reaches the conversion as an fp32 number whose last bit
// stands for everything below it, so that nothing is lost before it.  16-bit
// inputs would pay for that: 4096 x 14336 both ways 81 us against 57, bound by the
// vector unit instead of by memory.  What they give up: exact quotients stay clear of
// such a middle by far more than an fp32 rounding or lie on it, and where they
// lie on it the rounded scale moves some off it, to either side (one pair
// of bfloat16 significands in about 10^4; half a step of e4m3 either way).
#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

namespace {

constexpr double kE4m3Max = 448.0;
constexpr double kMinScale = 1.1754943508222875e-38;   // 2^-126

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Eight consecutive elements of one input type.
template <int TYPE>
struct Eight;   // 16-bit formats: four registers of two values

template <>
struct Eight<GEMM_TYPE_BF16> {
  static constexpr int BYTES = 16;
  u32x4 v;
  __device__ __forceinline__ void load(const uint8_t* p, int valid) {
    v = load8h_upto(reinterpret_cast<const uint16_t*>(p), valid);
  }
  __device__ __forceinline__ float at(int e) const {
    return __builtin_bit_cast(float, e & 1 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16);
  }
  // Magnitudes as packed pairs of 15-bit integers, and what a maximum of those
  // stands for.
  static constexpr int PARTS = 4;
  typedef u16x2 Mag;
  __device__ __forceinline__ Mag mag(int i) const {
    return __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu);
  }
  static __device__ __forceinline__ float value(uint32_t m) {
    return __builtin_bit_cast(float, m << 16);
  }
};
template <>
struct Eight<GEMM_TYPE_F16> : Eight<GEMM_TYPE_BF16> {
  __device__ __forceinline__ float at(int e) const {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(v[e / 2] >> (16 * (e & 1))));
  }
  static __device__ __forceinline__ float value(uint32_t m) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)m);
  }
};
template <>
struct Eight<GEMM_TYPE_F32> {
  static constexpr int BYTES = 32;
  u32x4 v[2];
  __device__ __forceinline__ void load(const uint8_t* p, int valid) {
    const uint32_t* f = reinterpret_cast<const uint32_t*>(p);
    if (valid >= 8) {
      v[0] = load16(p);
      v[1] = load16(p + 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e / 4][e % 4] = e < valid ? f[e] : 0u;
    }
  }
  __device__ __forceinline__ float at(int e) const {
    return __builtin_bit_cast(float, (uint32_t)v[e / 4][e % 4]);
  }
  static constexpr int PARTS = 8;
  typedef uint32_t Mag;
  __device__ __forceinline__ Mag mag(int i) const { return v[i / 4][i % 4] & 0x7fffffffu; }
  static __device__ __forceinline__ float value(uint32_t m) { return __builtin_bit_cast(float, m); }
};

__device__ __forceinline__ u16x2 mag_max(u16x2 a, u16x2 b) { return __builtin_elementwise_max(a, b); }
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t mag_all(u16x2 a) { return a[0] > a[1] ? a[0] : a[1]; }
__device__ __forceinline__ uint32_t mag_all(uint32_t a) { return a; }

// Maximum over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
#define LASG_ROR(n) \
  x = mag_max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + n, 0xf, 0xf, false))
  LASG_ROR(8);
  LASG_ROR(4);
  LASG_ROR(2);
  LASG_ROR(1);
#undef LASG_ROR
  return x;
}

// A block's scale, and what its quotients need.  (An infinite or NaN scale takes
// no remainder step: infinity times zero.)
template <int TYPE>
struct Scale {
  float s, r, sc;
  __device__ __forceinline__ explicit Scale(float amax) {
    s = amax / (float)kE4m3Max;
    if (s < (float)kMinScale) s = (float)kMinScale;   // (false for NaN)
    r = 1.0f / s;
    sc = __builtin_fabsf(s) < __builtin_inff() ? s : 0.0f;
  }
  // Eight values become their quotients.
  __device__ __forceinline__ void operator()(float (&x)[8]) const {
    float by = r, of = sc;
    if constexpr (TYPE == GEMM_TYPE_BF16) {
      // (A branch that is seldom taken: 2^-126, the scale of zeros and of what lies past
      // the end, divides exactly.  Without it small calls took up to 5 % longer.)
      const bool tiny = s < 0x1p-60f && s != (float)kMinScale;
      if (__builtin_expect(__any(tiny), 0)) {
        const float up = tiny ? 0x1p64f : 1.0f;
        by = 1.0f / (s * up);
        of *= up;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= up;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = x[e] * by;
      x[e] = __builtin_fmaf(-__builtin_fmaf(q, of, -x[e]), by, q);
    }
  }
};
template <>
struct Scale<GEMM_TYPE_F32> {
  // x / s as 7 x / (7 s): 448 = 7 x 64, so that both are exact in 64 bits.
  static constexpr double kPart = 7.0;
  float s;
  double r, sc;
  __device__ __forceinline__ explicit Scale(float amax) {
    double s7 = (double)amax * (kPart / kE4m3Max);
    if (s7 < kPart * kMinScale) s7 = kPart * kMinScale;
    s = (float)(s7 * (1.0 / kPart));
    r = 1.0 / s7;
    sc = s7 <= 3.5e38 ? s7 : 0.0;
  }
  __device__ __forceinline__ void operator()(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = quotient(x[e]);
  }
  __device__ __forceinline__ float quotient(float x) const {
    const double x7 = kPart * (double)x, q0 = x7 * r;
    const double q = __builtin_fma(-__builtin_fma(q0, sc, -x7), r, q0);
    const uint64_t bits = __builtin_bit_cast(uint64_t, q);
    const uint32_t lo = (uint32_t)bits, below = lo & 0x1fffffffu;   // what fp32 does not hold
    const uint32_t odd = (lo & 0xe0000000u) | (below != 0 ? 0x20000000u : 0u);
    return (float)__builtin_bit_cast(double, (bits & 0xffffffff00000000u) | odd);
  }
};

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

__device__ __forceinline__ void store8_upto(uint8_t* p, u32x2 v, int valid) {
  if (valid >= 8) {
    *reinterpret_cast<u32x2_any*>(p) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = (uint8_t)(v[e / 4] >> (8 * (e % 4)));
  }
}

}  // namespace

// One scale per row and block of 128 columns, no transpose: 16 lanes take one
// such block, eight columns each, and a wave 16 rows of one block of columns.
// Bound by memory; with few rows by the latency of one load, a wave reduction
// and one store (8 x 4096 bfloat16: 3.1 us, the time of an empty launch and a load).
template <int TYPE>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantizeCall p) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int kbs = (int)(((unsigned)p.cols + kBlockK - 1) / kBlockK);
  for (int kb = blockIdx.x; kb < kbs; kb += gridDim.x) {
    const int64_t col = (int64_t)kb * kBlockK + 8 * (lane % 16);
    const int valid = (int)(p.cols - col);
    for (int64_t r0 = (int64_t)blockIdx.y * 64 + 16 * wave; r0 < p.rows;
         r0 += (int64_t)gridDim.y * 64) {
      Eight<TYPE> x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = r0 + 4 * i + lane / 16;
        const int64_t rr = row < p.rows ? row : p.rows - 1;
        x[i].load(static_cast<const uint8_t*>(p.X) +
                      (rr * p.ldx + col) * (Eight<TYPE>::BYTES / 8), valid);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = r0 + 4 * i + lane / 16;
        typename Eight<TYPE>::Mag m = x[i].mag(0);
#pragma unroll
        for (int e = 1; e < Eight<TYPE>::PARTS; ++e) m = mag_max(m, x[i].mag(e));
        const Scale<TYPE> sc(Eight<TYPE>::value(max16(mag_all(m))));
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = x[i].at(e);
        sc(q);
        if (row < p.rows) {
          const u32x2 v = {pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
          store8_upto(p.Q + row * p.ldq + col, v, valid);
          if (lane % 16 == 0) p.S[(int64_t)kb * p.lds + row] = sc.s;
        }
      }
    }
  }
}

// Everything else: a workgroup takes a 128 x 128 tile, one read of which gives
// the scales and values along rows, along columns, or of the whole block.
// Thread (g, c) holds rows 8 g .. + 7 of columns 8 c .. + 7, so that a row's
// maximum is one over 16 neighbouring lanes, a column's one over the threads of
// equal c (two wave steps and one exchange through LDS), and both byte orders
// come out of the conversion by itself: pairs along the row for the matrix,
// pairs along the column for its transpose, which crosses LDS as 8-byte pieces
// (slot g of column j of chunk c lies at g ^ c, which spreads the writes over
// the banks) and leaves in whole 128-byte rows.
// Bound by memory: 4096 x 14336 bfloat16 both ways 57 us (4.1 TB/s, a copy reaches
// 5.1; the vector unit is busy 59 %), 4096 x 4096 fp32 in 128 x 128 blocks both ways
// 18.5 to 20 (5.0 and more).
// PLAIN / TURNED: which of the two are wanted; BLOCK: one scale per 128 x 128.
template <int TYPE, bool PLAIN, bool TURNED, bool BLOCK>
__global__ void __launch_bounds__(256) quantize_tile_kernel(QuantizeCall p) {
  __shared__ __attribute__((aligned(16))) uint8_t turned[TURNED ? 128 * 128 : 16];
  __shared__ uint32_t maxima[4][128];
  const int tid = threadIdx.x, wave = tid / kWave;
  const int g = tid / 16, c = tid % 16;
  const int tiles_n = (int)(((unsigned)p.cols + 127) / 128);
  const int tiles_m = (int)(((unsigned)p.rows + 127) / 128);
  typedef Eight<TYPE> E;
  for (int tm = blockIdx.y; tm < tiles_m; tm += gridDim.y)
    for (int tn = blockIdx.x; tn < tiles_n; tn += gridDim.x) {
      const int rows = p.rows - tm * 128 < 128 ? p.rows - tm * 128 : 128;
      const int cols = p.cols - tn * 128 < 128 ? p.cols - tn * 128 : 128;
      const int64_t row0 = (int64_t)tm * 128 + 8 * g;
      const int64_t col0 = (int64_t)tn * 128 + 8 * c;
      const int vr = rows - 8 * g, vc = cols - 8 * c;   // rows and columns there are
      E x[8];
      {
        const uint8_t* src = static_cast<const uint8_t*>(p.X) +
                             (row0 * p.ldx + col0) * (E::BYTES / 8);
        const int64_t step = (int64_t)p.ldx * (E::BYTES / 8);
        if (rows == 128 && cols == 128) {   // (uniform: no bounds in whole tiles)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i].load(src + i * step, 8);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i].load(src + i * step, i < vr ? vc : 0);
        }
      }
      typename E::Mag m;
      uint32_t row_max[8];
      typename E::Mag col_max[E::PARTS];
      if constexpr (PLAIN && !BLOCK) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m = x[i].mag(0);
#pragma unroll
          for (int e = 1; e < E::PARTS; ++e) m = mag_max(m, x[i].mag(e));
          row_max[i] = max16(mag_all(m));
        }
      }
      if constexpr (TURNED || BLOCK) {
#pragma unroll
        for (int e = 0; e < E::PARTS; ++e) {
          m = x[0].mag(e);
#pragma unroll
          for (int i = 1; i < 8; ++i) m = mag_max(m, x[i].mag(e));
          col_max[e] = m;
        }
      }
      if constexpr (BLOCK) {
        m = col_max[0];
#pragma unroll
        for (int e = 1; e < E::PARTS; ++e) m = mag_max(m, col_max[e]);
        uint32_t all = max16(mag_all(m));
        all = mag_max(all, (uint32_t)__shfl_xor((int)all, 16));
        all = mag_max(all, (uint32_t)__shfl_xor((int)all, 32));
        if (tid % kWave == 0) maxima[0][wave] = all;
        __syncthreads();
        uint32_t tile_max = maxima[0][0];
#pragma unroll
        for (int w = 1; w < 4; ++w) tile_max = mag_max(tile_max, maxima[0][w]);
        const Scale<TYPE> sc(E::value(tile_max));
        if (tid == 0) {
          if constexpr (PLAIN) p.S[(int64_t)tn * p.lds + tm] = sc.s;
          if constexpr (TURNED) p.ST[(int64_t)tm * p.ldst + tn] = sc.s;
        }
        float q[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) q[i][e] = x[i].at(e);
#pragma unroll
        for (int i = 0; i < 8; ++i) sc(q[i]);
        if constexpr (PLAIN) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const u32x2 v = {pack4(q[i][0], q[i][1], q[i][2], q[i][3]),
                             pack4(q[i][4], q[i][5], q[i][6], q[i][7])};
            if (i < vr) store8_upto(p.Q + (row0 + i) * p.ldq + col0, v, vc);
          }
        }
        if constexpr (TURNED) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const u32x2 v = {pack4(q[0][e], q[1][e], q[2][e], q[3][e]),
                             pack4(q[4][e], q[5][e], q[6][e], q[7][e])};
            *reinterpret_cast<u32x2*>(turned + (8 * c + e) * 128 + 8 * (g ^ c)) = v;
          }
        }
      } else {
        if constexpr (TURNED) {
          uint32_t cm[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (E::PARTS == 8)
              cm[e] = __builtin_bit_cast(uint32_t, col_max[e % E::PARTS]);
            else
              cm[e] = (__builtin_bit_cast(uint32_t, col_max[e / 2]) >> (16 * (e & 1))) & 0xffffu;
            cm[e] = mag_max(cm[e], (uint32_t)__shfl_xor((int)cm[e], 16));
            cm[e] = mag_max(cm[e], (uint32_t)__shfl_xor((int)cm[e], 32));
          }
          if (tid % kWave < 16) {
            *reinterpret_cast<u32x4*>(&maxima[wave][8 * c]) = u32x4{cm[0], cm[1], cm[2], cm[3]};
            *reinterpret_cast<u32x4*>(&maxima[wave][8 * c + 4]) = u32x4{cm[4], cm[5], cm[6], cm[7]};
          }
        }
        if constexpr (PLAIN) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const Scale<TYPE> sc(E::value(row_max[i]));
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = x[i].at(e);
            sc(q);
            const u32x2 v = {pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
            if (i < vr) {
              store8_upto(p.Q + (row0 + i) * p.ldq + col0, v, vc);
              if (c == 0) p.S[(int64_t)tn * p.lds + row0 + i] = sc.s;
            }
          }
        }
        if constexpr (TURNED) {
          __syncthreads();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t cmax = maxima[0][8 * c + e];
#pragma unroll
            for (int w = 1; w < 4; ++w) cmax = mag_max(cmax, maxima[w][8 * c + e]);
            const Scale<TYPE> sc(E::value(cmax));
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = x[i].at(e);
            sc(q);
            const u32x2 v = {pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
            *reinterpret_cast<u32x2*>(turned + (8 * c + e) * 128 + 8 * (g ^ c)) = v;
            if (g == 0 && e < vc) p.ST[(int64_t)tm * p.ldst + col0 + e] = sc.s;
          }
        }
      }
      if constexpr (TURNED) {
        __syncthreads();
        // Column j of the tile as a row of the transpose: eight threads, 16 bytes each.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = i * 32 + tid / 8, t = tid % 8;
          const int cc = j / 8;
          const u32x4 v = *reinterpret_cast<const u32x4*>(turned + j * 128 + 16 * (t ^ (cc >> 1)));
          const u32x4 w = cc & 1 ? u32x4{v[2], v[3], v[0], v[1]} : v;
          if (j < cols) {
            uint8_t* dst = p.QT + ((int64_t)tn * 128 + j) * p.ldqt + (int64_t)tm * 128 + 16 * t;
            const int left = rows - 16 * t;
            if (left >= 16) {
              *reinterpret_cast<u32x4_any*>(dst) = w;
            } else {
              store8_upto(dst, u32x2{w[0], w[1]}, left);
              store8_upto(dst + 8, u32x2{w[2], w[3]}, left - 8);
            }
          }
        }
      }
      __syncthreads();   // the next tile reuses the LDS arrays
    }
}

namespace {

template <int TYPE>
hipError_t launch_quantize_as(const QuantizeCall& c, hipStream_t s) {
  const unsigned kbs = ((unsigned)c.cols + 127) / 128;
  const unsigned rbs = ((unsigned)c.rows + 127) / 128;
  const dim3 tiles(kbs < (1u << 20) ? kbs : (1u << 20), rbs < 32768u ? rbs : 32768u);
  const bool plain = c.Q != nullptr, turned = c.QT != nullptr;
  if (c.block_rows == 1) {
    if (!turned) {
      const unsigned rgs = ((unsigned)c.rows + 63) / 64;
      const dim3 grid(tiles.x, rgs < 32768u ? rgs : 32768u);
      quantize_rows_kernel<TYPE><<<grid, 256, 0, s>>>(c);
    } else if (plain) {
      quantize_tile_kernel<TYPE, true, true, false><<<tiles, 256, 0, s>>>(c);
    } else {
      quantize_tile_kernel<TYPE, false, true, false><<<tiles, 256, 0, s>>>(c);
    }
  } else if (plain && turned) {
    quantize_tile_kernel<TYPE, true, true, true><<<tiles, 256, 0, s>>>(c);
  } else if (plain) {
    quantize_tile_kernel<TYPE, true, false, true><<<tiles, 256, 0, s>>>(c);
  } else {
    quantize_tile_kernel<TYPE, false, true, true><<<tiles, 256, 0, s>>>(c);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const QuantizeCall& c, hipStream_t s) {
  switch (c.type) {
    case GEMM_TYPE_F32: return launch_quantize_as<GEMM_TYPE_F32>(c, s);
    case GEMM_TYPE_F16: return launch_quantize_as<GEMM_TYPE_F16>(c, s);
    default: return launch_quantize_as<GEMM_TYPE_BF16>(c, s);
  }
}

}  // namespace lasg
