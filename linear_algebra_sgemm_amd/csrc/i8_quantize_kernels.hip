// Quantisation of rows to int8: for every row the scale s = max(max|x| / 127,
// 2^-126) and the whole numbers nearest to x / s (ties to even), s and x / s
// rounded to fp32.  The operands of the int8 product, tokens and channels alike.
//
// Magnitudes are compared as the integers of their bits without the sign, an order
// in which NaN is above infinity: a row that holds one has a NaN or infinite scale,
// and zeros for its values, whose product with such a scale is NaN.
//
// The quotient is formed from the correctly rounded reciprocal r of s: q0 = x r, q
// = q0 + r (x - q0 s) with fused multiply-adds, which is x / s correctly rounded
// (Markstein's theorem) unless the remainder underflows.  Below s = 2^-60, which binary16
// does not reach, x and s are multiplied by 2^64 first, exactly.  q + 1.5 x 2^23 holds the
// nearest whole number, ties to even, in its last bits: the byte.
//
// Memory bounds it: a row is read once, into registers, by a wave, a workgroup of
// 256 or one of 1024 threads (longer rows are read again from the caches).  4096 x 14336
// bfloat16 32 us (5.5 TB/s), 4096 x 4096 fp32 13.6; 8 x 4096 4.4, the launch.
#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

namespace {

constexpr float kMinRowScale = 0x1p-126f;
constexpr int kMostGroups = 1 << 20;   // of a launch; further rows in a loop
constexpr float kWhole = 12582912.0f;   // 1.5 x 2^23

typedef uint32_t u32_any __attribute__((aligned(1)));

// 16 bytes of a row: eight 16-bit values or four fp32 ones.
template <int TYPE>
struct Chunk16 {
  static constexpr int N = 8, SIZE = 2;
  static __device__ __forceinline__ float at(u32x4 v, int e) {
    const uint16_t b = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    return TYPE == GEMM_TYPE_F16 ? LmF16::value(b) : LmBF16::value(b);
  }
  // Largest magnitude as the bits of an fp32 number.
  static __device__ __forceinline__ uint32_t most(u32x4 v, uint32_t m) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = v[e] & 0x7fff7fffu, hi = x >> 16, lo = x & 0xffffu;
      const uint32_t h = hi > lo ? hi : lo;
      m = m > h ? m : h;
    }
    return m;
  }
  static __device__ __forceinline__ float magnitude(uint32_t m) {
    return TYPE == GEMM_TYPE_F16 ? LmF16::value((uint16_t)m) : LmBF16::value((uint16_t)m);
  }
};
template <>
struct Chunk16<GEMM_TYPE_F32> {
  static constexpr int N = 4, SIZE = 4;
  static __device__ __forceinline__ float at(u32x4 v, int e) {
    return __builtin_bit_cast(float, (uint32_t)v[e]);
  }
  static __device__ __forceinline__ uint32_t most(u32x4 v, uint32_t m) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = v[e] & 0x7fffffffu;
      m = m > x ? m : x;
    }
    return m;
  }
  static __device__ __forceinline__ float magnitude(uint32_t m) {
    return __builtin_bit_cast(float, m);
  }
};

// Maximum over a wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t y = (uint32_t)__shfl_xor((int)x, d);
    x = x > y ? x : y;
  }
  return x;
}

struct RowScale {
  float s, up, su, r;
  bool finite;
  __device__ __forceinline__ explicit RowScale(float most) {
    s = most / 127.0f;
    finite = s < __builtin_inff();   // (false for NaN)
    if (s < kMinRowScale) s = kMinRowScale;
    up = s < 0x1p-60f ? 0x1p64f : 1.0f;
    su = s * up;
    r = 1.0f / su;
  }
  __device__ __forceinline__ uint32_t byte(float x) const {
    x *= up;
    const float q0 = x * r;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, su, x), r, q0);
    return __builtin_bit_cast(uint32_t, q + kWhole);
  }
};

// Four numbers' last bytes.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
  return lo | hi << 16;
}

// Where a thread's chunk begins that would begin at `col`: the last chunk of a row is
// its last N values (those that it shares with the one before come out the same).
template <int TYPE>
__device__ __forceinline__ int begin_of(int col, int cols) {
  return col < cols - Chunk16<TYPE>::N ? col : cols - Chunk16<TYPE>::N;
}

template <int TYPE>
__device__ __forceinline__ u32x4 get(const uint8_t* row, int col, int cols) {
  typedef Chunk16<TYPE> C;
  if (cols < C::N) return load16_row(row, 0, cols * C::SIZE);   // (zeros behind)
  return load16(row + (int64_t)begin_of<TYPE>(col, cols) * C::SIZE);
}

template <int TYPE>
__device__ __forceinline__ void put(const RowScale& sc, u32x4 v, int8_t* q, int col, int cols) {
  typedef Chunk16<TYPE> C;
  uint32_t w[C::N / 4];
#pragma unroll
  for (int h = 0; h < C::N / 4; ++h) {
    w[h] = pack4(sc.byte(C::at(v, 4 * h)), sc.byte(C::at(v, 4 * h + 1)),
                 sc.byte(C::at(v, 4 * h + 2)), sc.byte(C::at(v, 4 * h + 3)));
    if (!sc.finite) w[h] = 0u;
  }
  if (col >= cols) return;
  if (cols < C::N) {
#pragma unroll
    for (int e = 0; e < C::N; ++e)
      if (e < cols) q[e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
    return;
  }
  q += begin_of<TYPE>(col, cols);   // (stored past the caches: 16384 x 2048 binary16 20 -> 17 us)
  if constexpr (C::N == 8)
    __builtin_nontemporal_store(u32x2{w[0], w[C::N / 4 - 1]}, reinterpret_cast<u32x2_any*>(q));
  else
    __builtin_nontemporal_store(w[0], reinterpret_cast<u32_any*>(q));
}

}  // namespace

// THREADS of a workgroup's 256 (or all of 1024) for a row, CHUNKS of 16 bytes each.
template <int TYPE, int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS > 256 ? THREADS : 256)
i8_quantize_kernel(I8QuantizeCall p) {
  typedef Chunk16<TYPE> C;
  constexpr int BLOCK = THREADS > 256 ? THREADS : 256, ROWS = BLOCK / THREADS;
  constexpr int WAVES = THREADS / kWave;
  __shared__ uint32_t part[WAVES > 1 ? WAVES : 1];
  const int at = threadIdx.x % THREADS;
  // (With more than one wave a row, a workgroup has one row and its waves stay together.)
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS; row < p.rows;
       row += (int64_t)gridDim.x * ROWS) {
    const uint8_t* x = static_cast<const uint8_t*>(p.X) + row * p.ldx * C::SIZE;
    u32x4 v[CHUNKS];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) v[i] = get<TYPE>(x, (i * THREADS + at) * C::N, p.cols);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) m = C::most(v[i], m);
    m = wave_max(m);
    if constexpr (WAVES > 1) {
      if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) m = m > part[w] ? m : part[w];
      __syncthreads();
    }
    const RowScale sc(C::magnitude(m));
    if (at == 0) p.S[row] = sc.s;
    int8_t* q = p.Q + row * p.ldq;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) put<TYPE>(sc, v[i], q, (i * THREADS + at) * C::N, p.cols);
  }
}

// Rows of any length: read twice.
template <int TYPE>
__global__ void __launch_bounds__(1024) i8_quantize_long_kernel(I8QuantizeCall p) {
  typedef Chunk16<TYPE> C;
  __shared__ uint32_t part[16];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const uint8_t* x = static_cast<const uint8_t*>(p.X) + row * p.ldx * C::SIZE;
    uint32_t m = 0;
#pragma unroll 4
    for (int col = threadIdx.x * C::N; col < p.cols; col += 1024 * C::N)
      m = C::most(get<TYPE>(x, col, p.cols), m);
    m = wave_max(m);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) m = m > part[w] ? m : part[w];
    __syncthreads();
    const RowScale sc(C::magnitude(m));
    if (threadIdx.x == 0) p.S[row] = sc.s;
    int8_t* q = p.Q + row * p.ldq;
#pragma unroll 4
    for (int col = threadIdx.x * C::N; col < p.cols; col += 1024 * C::N)
      put<TYPE>(sc, get<TYPE>(x, col, p.cols), q, col, p.cols);
  }
}

namespace {

template <int TYPE, int THREADS, int CHUNKS>
hipError_t launch_rows(const I8QuantizeCall& c, hipStream_t s) {
  constexpr int BLOCK = THREADS > 256 ? THREADS : 256, ROWS = BLOCK / THREADS;
  const int64_t groups = ((int64_t)c.rows + ROWS - 1) / ROWS;
  const unsigned grid = (unsigned)(groups < kMostGroups ? groups : kMostGroups);
  i8_quantize_kernel<TYPE, THREADS, CHUNKS><<<grid, BLOCK, 0, s>>>(c);
  return hipGetLastError();
}

template <int TYPE, int THREADS>
hipError_t launch_threads(const I8QuantizeCall& c, int chunks, hipStream_t s) {
  const int each = (chunks + THREADS - 1) / THREADS;
  if (each <= 1) return launch_rows<TYPE, THREADS, 1>(c, s);
  if (each <= 2) return launch_rows<TYPE, THREADS, 2>(c, s);
  if (each <= 4) return launch_rows<TYPE, THREADS, 4>(c, s);
  return launch_rows<TYPE, THREADS, 8>(c, s);
}

template <int TYPE>
hipError_t launch_type(const I8QuantizeCall& c, int cus, hipStream_t s) {
  const int chunks = (c.cols + Chunk16<TYPE>::N - 1) / Chunk16<TYPE>::N;
  if (chunks > 8 * 1024) {
    i8_quantize_long_kernel<TYPE><<<c.rows < kMostGroups ? c.rows : kMostGroups, 1024, 0, s>>>(c);
    return hipGetLastError();
  }
  // A wave a row where that makes eight waves a CU, more threads where rows are few.
  const bool few = c.rows < 8 * cus;
  if (chunks <= (few ? 1 : 8) * 64) return launch_threads<TYPE, 64>(c, chunks, s);
  if (chunks <= (few ? 2 : 8) * 256) return launch_threads<TYPE, 256>(c, chunks, s);
  return launch_threads<TYPE, 1024>(c, chunks, s);
}

}  // namespace

hipError_t launch_i8_quantize(const I8QuantizeCall& c, int cus, hipStream_t s) {
  switch (c.type) {
    case GEMM_TYPE_F32: return launch_type<GEMM_TYPE_F32>(c, cus, s);
    case GEMM_TYPE_F16: return launch_type<GEMM_TYPE_F16>(c, cus, s);
    default: return launch_type<GEMM_TYPE_BF16>(c, cus, s);
  }
}

}  // namespace lasg
