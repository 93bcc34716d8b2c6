// The int8 product with a scale for every token and channel:
//     u[m][n] = alpha sa[m] sb[n] sum_k A[m][k] B[n][k] + bias[n],   C = act(u),
// or with a gate (B has 2 N rows)  C[m][n] = act(u[m][n]) u[m][N + n];  A (M x K)
// and B (N x K) in int8, both contiguous along K.  Grouped: the rows of A are those of
// one group after the other, and B, sb and bias are their group's.
//
// The sums are int32 and exact (K <= 131071: 2^17 products of -128 and -128 would
// pass 2^31 - 1), so neither the order nor the split of K changes a result.
// Each is rounded to fp32 once, then scaled.
//
// Operand k order: an MFMA pairs the same lane and byte of both operands, so
// any assignment of k to lanes serves if both use it.
#include "i8_common.h"

namespace lasg {

namespace {

// One 16-row fragment of 128 k: lane l holds row l % 16, the 16-byte chunks
// l / 16 and l / 16 + 4 of its eight.
struct Frag8 {
  u32x4 c[2];
};

__device__ __forceinline__ void load_frag(Frag8& f, const int8_t* row, int lane, int k0) {
  const int k = k0 + 16 * (lane / 16);
  f.c[0] = load16(row + k);
  f.c[1] = load16(row + k + 64);
}
// The same at the end of a row of K bytes.
__device__ __forceinline__ void load_frag_tail(Frag8& f, const int8_t* row, int lane, int k0, int K) {
  const int k = k0 + 16 * (lane / 16);
  f.c[0] = load16_row(row, k, K);
  f.c[1] = load16_row(row, k + 64, K);
}

__device__ __forceinline__ i32x4 add_product(const Frag8& x, const Frag8& y, i32x4 acc) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x.c[h]),
                                                __builtin_bit_cast(i32x4, y.c[h]), acc, 0, 0, 0);
  return acc;
}

// Four consecutive values of one row of C (columns col ..; `left` of them exist).
__device__ __forceinline__ void store_c(const I8Call& p, int64_t row, int64_t col, f32x4 v) {
  const int64_t left = p.N - col;
  if (p.type == GEMM_TYPE_F32) {
    float* d = static_cast<float*>(p.C) + row * p.ldc + col;
    if (left >= 4) {
      *reinterpret_cast<f32x4_any*>(d) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) d[e] = v[e];
    }
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = p.type == GEMM_TYPE_F16 ? LmF16::bits(v[e]) : LmBF16::bits(v[e]);
  uint16_t* d = static_cast<uint16_t*>(p.C) + row * p.ldc + col;
  if (left >= 4) {
    *reinterpret_cast<u32x2_any*>(d) = __builtin_bit_cast(u32x2, h);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) d[e] = h[e];
  }
}

}  // namespace

// A tile of 16 MF rows of A by 16 NF rows of B per workgroup, its eight waves taking
// an eighth of the blocks of 128 k each, straight from memory into MFMA operands, the
// eight sums added in LDS at the end.  Any shape, stride and alignment.  Few rows:
// the bytes of B bound it, every one of which is read once; what matters is
// how many are on their way.  A wave loads GROUP blocks before it multiplies the first,
// and with many fragments the next block of B while it multiplies this one.
// With a gate the 16 rows of a fragment of B are eight of each half, so that
// a result's two sums lie 32 lanes apart in one fragment.
template <int MF, int NF, bool GROUPED>
__global__ void __launch_bounds__(512) i8_ksplit_kernel(I8Call p) {
  constexpr int GROUP = MF + NF <= 3 ? 4 : MF * NF <= 4 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) i32x4 part[4][MF * NF][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane % 16, g = lane / 16;
  const int64_t b_rows = i8_b_rows(p);
  const unsigned tiles_n = (unsigned)((b_rows + 16 * NF - 1) / (16 * NF));
  const GroupTiles<16 * MF> tiles(p);
  const unsigned tiles_m = GROUPED ? (unsigned)tiles.total : ((unsigned)p.M + 16 * MF - 1) / (16 * MF);
  const int full = p.K / kBlockK;
  for (unsigned tm = blockIdx.y; tm < tiles_m; tm += gridDim.y)
    for (unsigned tn = blockIdx.x; tn < tiles_n; tn += gridDim.x) {
      int group = 0, m0 = (int)(tm * 16 * MF), m_end = p.M;
      if constexpr (GROUPED) {
        tiles.find(p, (int)tm, group, m0, m_end);
        if (m0 >= m_end) continue;
      }
      const int8_t* b_mat = p.B + group * b_rows * p.ldb;
      const float* sb_v = p.SB + group * b_rows;
      const float* bias_v = p.bias == nullptr ? nullptr : p.bias + group * b_rows;
      // The row of B behind row x of fragment j (past the end: the last; not stored).
      const auto b_row = [&](int j, int x) -> int64_t {
        const int64_t f = (int64_t)tn * NF + j;
        if (!p.gated) {
          const int64_t row = 16 * f + x;
          return row < p.N ? row : p.N - 1;
        }
        const int64_t row = 8 * f + x % 8;
        return (row < p.N ? row : p.N - 1) + (x >= 8 ? p.N : 0);
      };
      // (Rows are compared from m0 on: m0 plus the tile's height may pass 2^31.)
      const int rows = m_end - m0;
      const int8_t* ap[MF];
      const int8_t* bp[NF];
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int row = 16 * i + r < rows ? m0 + 16 * i + r : m_end - 1;
        ap[i] = p.A + i8_a_row(p, row) * p.lda;
      }
#pragma unroll
      for (int j = 0; j < NF; ++j) bp[j] = b_mat + b_row(j, r) * p.ldb;
      // What this wave needs at the end: it finishes fragment `wave`, a lane four columns of one row
      // (with a gate the lanes of the first half, whose counterparts are 32 lanes on).
      static_assert(MF * NF <= 8, "a fragment a wave");
      const int end_at = 16 * (wave / NF) + r, end_j = wave % NF;
      const int end_row = m0 + (end_at < rows ? end_at : 0);
      const bool ends = wave < MF * NF && end_at < rows && (!p.gated || g < 2);
      float sa = 0.0f, sb[2][4] = {}, bias[2][4] = {};
      if (ends) {
        if (p.K != 0) sa = p.SA[i8_a_row(p, end_row)];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (h == 1 && !p.gated) continue;
            const int64_t n = b_row(end_j, 4 * g + 8 * h + e);
            if (p.K != 0) sb[h][e] = sb_v[n];
            if (bias_v != nullptr) bias[h][e] = bias_v[n];
          }
      }
      i32x4 sums[MF * NF];
#pragma unroll
      for (int f = 0; f < MF * NF; ++f) sums[f] = i32x4{0, 0, 0, 0};
      // (B first: the lane then holds four columns of one row of C)
      const auto multiply = [&](const Frag8 (&a)[MF], const Frag8 (&b)[NF])
          __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int j = 0; j < NF; ++j) sums[i * NF + j] = add_product(b[j], a[i], sums[i * NF + j]);
      };
      const auto load_a = [&](Frag8 (&a)[MF], int k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MF; ++i) load_frag(a[i], ap[i], lane, k0);
      };
      const auto load_b = [&](Frag8 (&b)[NF], int k0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NF; ++j) load_frag(b[j], bp[j], lane, k0);
      };
      const int first = (int)((int64_t)full * wave / 8), end = (int)((int64_t)full * (wave + 1) / 8);
      if constexpr (GROUP > 1) {
        for (int kb = first; kb < end; kb += GROUP) {
          Frag8 a[GROUP][MF], b[GROUP][NF];
#pragma unroll
          for (int u = 0; u < GROUP; ++u) {
            const int at = kb + u < end ? kb + u : end - 1;   // (an extra read, not used)
            load_b(b[u], at * kBlockK);
            load_a(a[u], at * kBlockK);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int u = 0; u < GROUP; ++u)
            if (kb + u < end) multiply(a[u], b[u]);
        }
      } else if (first < end) {
        Frag8 b[2][NF];
        load_b(b[0], first * kBlockK);
        // Two blocks a turn, so that the buffers of B keep their registers.
        for (int kb = first; kb < end; kb += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (kb + u >= end) break;
            Frag8 a[MF];
            load_a(a, (kb + u) * kBlockK);
            load_b(b[1 - u], (kb + u + 1 < end ? kb + u + 1 : kb + u) * kBlockK);
            __builtin_amdgcn_sched_barrier(0);
            multiply(a, b[u]);
          }
        }
      }
      if (full * kBlockK < p.K && wave == 7) {   // the last, shorter block
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          Frag8 b;
          load_frag_tail(b, bp[j], lane, full * kBlockK, p.K);
#pragma unroll
          for (int i = 0; i < MF; ++i) {
            Frag8 a;
            load_frag_tail(a, ap[i], lane, full * kBlockK, p.K);
            sums[i * NF + j] = add_product(b, a, sums[i * NF + j]);
          }
        }
      }
      // Waves 4 to 7 put their sums down, waves 0 to 3 add theirs (half the space).
      if (wave >= 4) {
#pragma unroll
        for (int f = 0; f < MF * NF; ++f) part[wave - 4][f][lane] = sums[f];
      }
      __syncthreads();
      if (wave < 4) {
#pragma unroll
        for (int f = 0; f < MF * NF; ++f) part[wave][f][lane] += sums[f];
      }
      __syncthreads();
      if (ends) {
        const SplitScale ma(sa, p.alpha_e);
        const auto value = [&](int h) __attribute__((always_inline)) {
          const int l = lane + 32 * h;
          const i32x4 v = (part[0][wave][l] + part[1][wave][l]) + (part[2][wave][l] + part[3][wave][l]);
          f32x4 u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const SplitScale mb(sb[h][e]);
            u[e] = i8_scaled(v[e], ma.m, ma.e, mb.m, mb.e, p.alpha, bias[h][e]);
          }
          return u;
        };
        f32x4 v = value(0);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = apply_act(v[e], p.act);
        int64_t col = ((int64_t)tn * NF + end_j) * 16 + 4 * g;
        if (p.gated) {
          const f32x4 u = value(1);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= u[e];
          col = ((int64_t)tn * NF + end_j) * 8 + 4 * g;
        }
        if (col < p.N) store_c(p, end_row, col, v);
      }
      __syncthreads();   // the next tile reuses the LDS array
    }
}

namespace {

template <int MF, int NF>
hipError_t launch_ksplit(const I8Call& c, hipStream_t s) {
  const int64_t tn = (i8_b_rows(c) + 16 * NF - 1) / (16 * NF), tm = i8_tiles_m(c, 16 * MF);
  const dim3 grid((unsigned)(tn < (1 << 20) ? tn : 1 << 20), (unsigned)(tm < 32768 ? tm : 32768));
  if (c.groups > 0)
    i8_ksplit_kernel<MF, NF, true><<<grid, 512, 0, s>>>(c);
  else
    i8_ksplit_kernel<MF, NF, false><<<grid, 512, 0, s>>>(c);
  return hipGetLastError();
}

}  // namespace

namespace {

// Groups that have rows, and rows of such a group, as if rows were spread at random.
struct Spread {
  double active, each;
  explicit Spread(const I8Call& c) {
    const double rows = c.M, groups = c.groups > 0 ? c.groups : 1;
    active = c.groups > 0 ? groups * (1 - __builtin_exp(-rows / groups)) : 1;
    each = rows / active;
  }
};

struct Tile {
  int m, n, per_cu;
  double one, every, all;   // see the rule
};
const Tile kTiles[7] = {{256, 256, 1, 1250, 1840, 1840}, {128, 256, 2, 970, 1140, 1910},
                        {128, 128, 2, 700, 760, 1130},   {64, 128, 2, 440, 470, 750},
                        {64, 64, 2, 320, 330, 480},      {32, 128, 2, 350, 360, 540},
                        {128, 128, 2, 1420, 1500, 1910}};

// Whether tiles of `m` rows read B once, and at least 96 MB of it: then it is copied past the caches.
// That is better where other weights are used before this one comes again, as in a model of many layers, and
// worse where the next call uses it too, which up to about 250 MB finds it in the last-level cache.  In
// us, without and with, other weights between | the same at once (64 x 128 and 32 x 128 tiles):
//   64 rows by 20480 x 4096 (84 MB)   24.5, 21.6 | 15.4, 20.3      36864 (151 MB)  41.8, 37.7 | 29.8, 36.1
//   by 28672 x 4096 (117 MB)          28.1, 23.7 | 19.7, 22.3      61440 (252 MB)  51.2, 43.4 | 36.9, 41.8
//   4 tokens on 64 experts (25 used): of 1024 x 4096 (111 MB)      23.2, 20.6 | 17.8, 17.8
//                                     of 2048 x 4096 (222 MB)      40.5, 36.3 | 30.5, 32.9
// A call does not say what comes between.  That weights of 96 MB and more have others between them,
// and smaller ones may not, is a guess: those would gain as well (61 MB 22.6, 20.5) and lose more (14.7, 19.1).
// Groups count as read once while nearly all fit one tile: rows spread at random vary by the root of
// their mean, so that at a mean of 0.7 x 32 two deviations more are 32.
bool reads_once(const I8Call& c, int m) {
  const Spread x(c);
  return x.active * (double)i8_b_rows(c) * c.K >= 96e6 && x.each <= (c.groups > 0 ? 0.7 : 1.0) * m;
}

}  // namespace

// The rule takes the tile of the least estimated time.  Measured on 256 CUs:
//  * tiles through LDS take a time per block of K that depends on how many of them
//    run, not on the shape: kTiles has it in ns for one of them, for one on every CU and for as
//    many as fit a CU.  4096 x 4096 x 4096: 256 x 256 62 us, 128 x 256 65, 128 x 128 73; 4096 x 14336 x
//    4096, 3.5 rounds of either: 241 and 228; 1024 x 4096 x 4096: 128 x 128 26, 128 x 256 33; 1024
//    x 1024 x 4096: 64 x 64 11.1, 64 x 128 14.8, 128 x 128 23.9.
//  * where the weights bound a call it takes their bytes at 5.5 TB/s (6.3 past the caches), and the
//    bytes that the CUs load at 40: 4 tokens on 64 experts of 2048 x 4096 32 x 128 tiles 37 us, 64
//    x 64 40; 64 rows by 28672 x 4096 64 x 128 22.6, 64 x 64 25, 32 x 128 29.
//  * K-split tiles of m x n take (m + n) K bytes through a CU's load path at 23 bytes a ns: 1 x
//    4096 x 4096 16 x 16 6.4 us, 64 x 64 through LDS 10.6; off 16-byte boundaries about 2.5 times
//    that (64 x 4096 x 4095: 32 x 32 34 us, 128 x 128 through registers 49; 128 x 4096: 64 x 32 52, 48).
int i8_tile(const I8Call& c, int cus, int force) {
  static const int kSplit[5][2] = {{64, 32}, {32, 32}, {32, 16}, {16, 32}, {16, 16}};
  const int64_t b_rows = i8_b_rows(c);
  // 32-bit row, column and tile numbers in the tiled kernels, and fewer than 2^32 threads a launch.  (A
  // larger call takes K-split tiles: 131328 x 131072 x 4096 472 ms, 130816 x 131072 x 4096 66.5.)
  const bool tiled = c.M <= (1 << 30) && b_rows <= (1 << 30) &&
                     i8_tiles_m(c, 32) * ((b_rows + 63) / 64) < (1 << 23);
  const bool direct = i8_direct(c);
  int tile = force;
  if (tile < 0) {
    const Spread x(c);
    // (Groups of 0.7 m rows take one tile, as in reads_once; of longer ones the last is half full.)
    const auto tiles = [&](int m, int n) {
      const double down = c.groups == 0      ? __builtin_ceil((double)c.M / m)
                          : x.each <= 0.7 * m ? 1
                                              : x.each / m + 0.5;
      return x.active * down * (double)((b_rows + n - 1) / n);
    };
    const double weights = x.active * (double)b_rows * c.K;
    double best = 1e30;
    const auto offer = [&](int t, double cost) {
      if (cost < best) {
        best = cost;
        tile = t;
      }
    };
    for (int t = direct ? 0 : 6; tiled && t < (direct ? 6 : 7); ++t) {
      const Tile& k = kTiles[t];
      const double n = tiles(k.m, k.n), round = (double)k.per_cu * cus;
      const double full = __builtin_floor(n / round), left = n - full * round, on = left / cus;
      double last = on <= 1 ? k.one + on * (k.every - k.one) : k.every + (on - 1) * (k.all - k.every);
      if (left == 0) last = 0;
      // (after whole rounds a CU's only workgroup gains little from the others' absence)
      else if (full > 0 && k.per_cu == 1 && last < 0.85 * k.all) last = 0.85 * k.all;
      const double blocks = (double)((c.K + kBlockK - 1) / kBlockK) + 2;   // (2: start and end)
      const double work = blocks * (full * k.all + last);
      const double bytes = weights / (reads_once(c, k.m) ? 6300 : 5500) + n * (k.m + k.n) * c.K / 40000;
      offer(t, work > bytes ? work : bytes);
    }
    for (int i = 0; i < 5; ++i) {
      const int m = kSplit[i][0], n = kSplit[i][1];
      const double rounds = __builtin_ceil(tiles(m, n) / cus);
      offer(7 + i, rounds * (m + n) * ((double)c.K + 512) / (direct ? 23 : 9));
    }
  }
  if (tile < 7 && !tiled) tile = 7;
  if (tile < 6 && !direct) tile = 6;
  return tile;
}

hipError_t launch_i8_gemm(const I8Call& c, int cus, int force, hipStream_t s) {
  const int tile = i8_tile(c, cus, force);
  switch (tile) {
    case 7: return launch_ksplit<4, 2>(c, s);
    case 8: return launch_ksplit<2, 2>(c, s);
    case 9: return launch_ksplit<2, 1>(c, s);
    case 10: return launch_ksplit<1, 2>(c, s);
    case 11: return launch_ksplit<1, 1>(c, s);
    default: return launch_i8_tile(c, tile, reads_once(c, kTiles[tile].m), s);
  }
}

}  // namespace lasg
