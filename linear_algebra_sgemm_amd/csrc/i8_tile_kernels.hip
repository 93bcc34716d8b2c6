// The int8 product in output tiles staged through LDS (formula: i8_kernels.hip),
// for outputs large enough that the matrix units bound it.
//
// A K tile is 128 columns: rows of 128 bytes, copied from memory straight into LDS
// (16 bytes a lane, whole 128-byte lines) STAGES tiles ahead.  Row r's eight 16-byte
// chunks lie permuted by (r / 2) % 8, so that the fragment reads of 16 neighbouring rows
// fall into 16 different bank groups.
//
// A wave multiplies 32x32 blocks, 32 columns of K a step, four steps a K tile: a step's
// fragments are read while the step before is multiplied, those of the next K
// tile's first step too, so a K tile has one meeting of the waves, before its last
// step: there all have read tile t whole (its stage takes tile t + STAGES from then on) and
// tile t + 1 has landed.  B is the first operand, so a lane holds the columns 8 q +
// 4 (lane / 32) + 0..3 of one row of C.  With a gate, every 32 rows of B in the tile are
// 16 of the first half and 16 of the second, so that both sums of a result
// are one lane's.
//
// What bounds it: for large outputs the power limit: 4096 x 4096 x 4096 in 256 x 256 tiles 61 us
// (2250 TOP/s) and 8192^3 452 (2430) at 1.65 GHz with the matrix unit busy 66 % of the
// cycles, where a library's int8 product reaches 2075 to 2170 TOP/s; the waves' fragment
// reads and the copies fill LDS's 128 bytes a cycle meanwhile.  4096 x 14336 x 4096 with bias and
// GELU 237 to 249 us.  For few rows the weights' bytes: 4 tokens on 64 experts of 2048 x
// 4096 37 us (6.0 TB/s), 64 x 28672 x 4096 22.5 (5.3 TB/s).  Few tiles with a long K: what a wave does
// for a K tile one after the other (fragment reads, a step's MFMAs on one block, the meeting).  64 x 4096 x
// 4096 takes 11.1 us, 4 of them its start and end and 0.225 every K tile; the same loop without its
// copies 9.4, without its MFMAs too 7.8; its matrix units are busy 15 % of the cycles, its waves wait 58 %.
// With several tiles on a CU the copies into LDS count as well, at 25 to 32 bytes a cycle and CU: 512 x 4096
// x 4096 17.0, without copies 11.9; 1024 x 4096 x 4096 in 128 x 128 tiles 26.4 and 18.0.
#include <type_traits>

#include "dma_common.h"
#include "i8_common.h"

namespace lasg {

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, bool DIRECT_, bool OWN_B_,
          bool GROUPED_, bool ONCE_>
struct I8Tile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int STAGES = STAGES_;
  static constexpr bool DIRECT = DIRECT_, GROUPED = GROUPED_;
  static constexpr bool ONCE = ONCE_;   // B is copied past the caches
  static constexpr int WAVES = WAVES_M * WAVES_N, THREADS = WAVES * kWave;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
  static constexpr int FM = WTM / 32, FN = WTN / 32, BLOCKS = FM * FN;
  // Waves side by side only: each copies and reads its own rows of B, so one stage of B
  // is enough (refilled once the wave holds its fragments).
  static constexpr bool OWN_B = OWN_B_;
  static_assert(!OWN_B || (WAVES_M == 1 && STAGES == 2 && DIRECT), "waves side by side");
  static constexpr int A_BYTES = BM * kBlockK, B_BYTES = BN * kBlockK;
  static constexpr int B_AT = STAGES * A_BYTES;
  static constexpr int STAGES_BYTES = B_AT + (OWN_B ? 1 : STAGES) * B_BYTES;
  static constexpr int A_LOADS = BM / 8 / WAVES, B_LOADS = BN / 8 / WAVES;   // per wave, 1 KiB each
  static constexpr int LOADS = A_LOADS + B_LOADS;
  // Epilogue: 32 rows of each wave's results, then the scales (split) and bias.
  static constexpr int REGION = 32 * WTN * 4;
  static constexpr int SCALES_AT = WAVES * REGION;
  static constexpr int EPILOGUE_BYTES = SCALES_AT + 4 * (3 * BN + 2 * BM);
  static constexpr int LDS_BYTES = STAGES_BYTES > EPILOGUE_BYTES ? STAGES_BYTES : EPILOGUE_BYTES;
  static_assert(DIRECT || STAGES == 2, "through registers one tile ahead");
  static_assert(STAGES >= 2 && (STAGES - 1) * LOADS <= 63, "copies on their way must fit vmcnt");
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "copies split evenly over waves");
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tile");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

struct I8TileArgs {
  I8Call c;
  int tiles_m, tiles_n, group_m;
  // K tiles that the tiles of one group (of a tile column) start behind those of the one
  // before.  All at the same K would read addresses a row apart, a power of two in most
  // weights, from a part of the memory channels only.
  int group_step, column_step;
};

namespace {

// dma16_sbase_u for lines that nobody else will read: they are not kept in the caches.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is listed as clobbered on purpose
__device__ __forceinline__ void dma16_sbase_once(const void* base, uint32_t offset, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
               :: "s"(__builtin_amdgcn_readfirstlane(lds_base)), "v"(offset), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop

template <class T>
struct I8Frags {
  i32x4 a[T::FM], b[T::FN];
};

// The results of a wave, 32 rows at a time: scales, bias, activation and gate in
// registers, rounded to C's type, through the wave's own piece of LDS (chunks permuted as
// above) so that whole rows are stored, 16 bytes a lane.
template <class T, int ACT, bool WIDE, bool GATED>
__device__ __forceinline__ void i8_write_back(const I8Call& c, const i32x16 (&sum)[T::FM][T::FN],
                                              uint8_t* lds, int wave, int m0, int m_end, int n0,
                                              int lane) {
  constexpr int WIDTH = GATED ? T::WTN / 2 : T::WTN;   // columns of C
  constexpr int SIZE = WIDE ? 4 : 2, ROW = WIDTH * SIZE, CHUNKS = ROW / 16;
  constexpr int LINE = ROW >= 256 ? 1 : 256 / ROW;     // rows in a line of the LDS banks
  static_assert(1024 % ROW == 0, "whole rows per store");
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const int l32 = lane % 32, half = lane / 32;
  uint8_t* region = lds + wave * T::REGION;
  const float* mb = reinterpret_cast<const float*>(lds + T::SCALES_AT) + wn * T::WTN + 4 * half;
  const int* eb = reinterpret_cast<const int*>(mb + T::BN);
  const float* bias = mb + 2 * T::BN;
  const float* ma = reinterpret_cast<const float*>(lds + T::SCALES_AT) + 3 * T::BN + wm * T::WTM + l32;
  const int* ea = reinterpret_cast<const int*>(ma + T::BM);
  const bool f16 = c.type == GEMM_TYPE_F16;
  const int col0 = n0 + wn * WIDTH;
  auto slot = [](int row, int chunk) {
    return row * ROW + 16 * (chunk ^ (row / LINE & (CHUNKS - 1)));
  };
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const float ma_i = ma[32 * i];
    const int ea_i = ea[32 * i];
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < (GATED ? 2 : 4); ++q) {
        // (`x`: columns x .. x + 3 of the fragment, whose sums are registers x / 2 ..)
        const auto scaled = [&](int x) __attribute__((always_inline)) {
          const f32x4 m4 = *reinterpret_cast<const f32x4*>(mb + 32 * j + x);
          const i32x4 e4 = *reinterpret_cast<const i32x4*>(eb + 32 * j + x);
          const f32x4 b4 = *reinterpret_cast<const f32x4*>(bias + 32 * j + x);
          f32x4 u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            u[e] = i8_scaled(sum[i][j][x / 2 + e], ma_i, ea_i, m4[e], e4[e], c.alpha, b4[e]);
          return u;
        };
        f32x4 v = scaled(8 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = apply_act(v[e], ACT);
        if constexpr (GATED) {
          const f32x4 u = scaled(8 * q + 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= u[e];
        }
        const int at = (GATED ? 16 : 32) * j + 8 * q + 4 * half;   // column in the wave's tile
        if constexpr (WIDE) {
          *reinterpret_cast<f32x4*>(region + slot(l32, at / 4)) = v;
        } else {
          uint16_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = f16 ? LmF16::bits(v[e]) : LmBF16::bits(v[e]);
          *reinterpret_cast<u32x2*>(region + slot(l32, at / 8) + 8 * half) =
              __builtin_bit_cast(u32x2, h);
        }
      }
    asm volatile("" ::: "memory");   // (one wave's LDS accesses keep their order)
    constexpr int ROWS = 1024 / ROW < 32 ? 1024 / ROW : 32;   // of a store
#pragma unroll
    for (int it = 0; it < 32 / ROWS; ++it) {
      const int r = it * ROWS + lane / CHUNKS, chunk = lane % CHUNKS;
      if (1024 / ROW > 32 && r >= 32) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(region + slot(r, chunk));
      const int row = m0 + wm * T::WTM + 32 * i + r, col = col0 + chunk * (16 / SIZE);
      if (row >= m_end || col >= c.N) continue;
      uint8_t* d = static_cast<uint8_t*>(c.C) + ((int64_t)row * c.ldc + col) * SIZE;
      if (col + 16 / SIZE <= c.N) {
        *reinterpret_cast<u32x4_any*>(d) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 16 / SIZE; ++e)
          if (col + e < c.N) {
            if constexpr (WIDE)
              reinterpret_cast<uint32_t*>(d)[e] = v[e % 4];
            else
              reinterpret_cast<uint16_t*>(d)[e] = (uint16_t)(v[e / 2 % 4] >> (16 * (e & 1)));
          }
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <class T, int ACT>
__device__ __forceinline__ void i8_write_as(const I8Call& c, const i32x16 (&sum)[T::FM][T::FN],
                                            uint8_t* lds, int wave, int m0, int m_end, int n0,
                                            int lane) {
  if (c.type == GEMM_TYPE_F32)
    c.gated ? i8_write_back<T, ACT, true, true>(c, sum, lds, wave, m0, m_end, n0, lane)
            : i8_write_back<T, ACT, true, false>(c, sum, lds, wave, m0, m_end, n0, lane);
  else
    c.gated ? i8_write_back<T, ACT, false, true>(c, sum, lds, wave, m0, m_end, n0, lane)
            : i8_write_back<T, ACT, false, false>(c, sum, lds, wave, m0, m_end, n0, lane);
}

}  // namespace

template <class T>
__global__ void __launch_bounds__(T::THREADS) __attribute__((amdgpu_waves_per_eu(2)))
i8_tile_kernel(I8TileArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS_BYTES];
  const I8Call& c = p.c;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const int l32 = lane % 32, half = lane / 32;
  const uint32_t lds_base = lds_offset(lds);
  const int b_rows = (int)i8_b_rows(c);
  int tile_m, tile_n, m0, m_end = c.M, group = 0;
  if constexpr (T::GROUPED) {
    const GroupTiles<T::BM> tiles(c);
    if ((int64_t)blockIdx.x >= (int64_t)tiles.total * p.tiles_n) return;
    tile_of_workgroup(blockIdx.x, tiles.total, p.tiles_n, p.group_m, tile_m, tile_n);
    tiles.find(c, tile_m, group, m0, m_end);
    if (m0 >= m_end) return;
  } else {
    tile_of_workgroup(blockIdx.x, p.tiles_m, p.tiles_n, p.group_m, tile_m, tile_n);
    m0 = tile_m * T::BM;
  }
  // First column of C; the tile's first row of B (of each half, with a gate).
  const int n0 = tile_n * (c.gated ? T::BN / 2 : T::BN);
  const int64_t group_b = (int64_t)group * b_rows;
  const int8_t* b_tile = c.B + (group_b + n0) * c.ldb;
  // Rows of A from where the tile begins, or anywhere in A.
  const int8_t* a_tile = c.index != nullptr ? c.A : c.A + (int64_t)m0 * c.lda;
  const int kts = (c.K + kBlockK - 1) / kBlockK;

  // The row of A (from a_tile) or B (from b_tile) that tile row `row` is; past the
  // end the last.
  auto a_row = [&](int row) __attribute__((always_inline)) {
    const int r = m0 + row < m_end ? row : m_end - 1 - m0;
    return c.index != nullptr ? i8_a_row(c, m0 + r) : (int64_t)r;
  };
  auto b_row = [&](int row) __attribute__((always_inline)) {
    const int at = c.gated ? row / 32 * 16 + row % 16 : row;
    const int r = n0 + at < c.N ? at : c.N - 1 - n0;
    return c.gated && (row & 16) ? r + c.N : r;
  };
  // Row (of the tile) and chunk that lane `l` copies in load v of this wave.
  auto slot = [&](int v, int l, int& row, int& chunk) __attribute__((always_inline)) {
    row = 8 * (v < T::A_LOADS ? wave * T::A_LOADS + v : wave * T::B_LOADS + v - T::A_LOADS) + l / 8;
    chunk = (l % 8) ^ ((row >> 1) & 7);
  };
  auto slot_at = [&](int v, int t) __attribute__((always_inline)) {
    return v < T::A_LOADS ? t % T::STAGES * T::A_BYTES + (wave * T::A_LOADS + v) * 1024
                          : T::B_AT + (T::OWN_B ? 0 : t % T::STAGES * T::B_BYTES) +
                                (wave * T::B_LOADS + v - T::A_LOADS) * 1024;
  };
  // K tiles in the order they are taken.  A last, shorter one goes through registers, with zeros
  // behind it; where whole ones are copied straight into LDS it is taken first, so that its
  // latency falls together with the first copies'.
  const bool tail_first = T::DIRECT && c.K % kBlockK != 0;
  const int whole = tail_first ? kts - 1 : kts;
  const int rotated = whole == 0 ? 0 : (int)(((unsigned)tile_n * p.column_step +
                                              (unsigned)group * p.group_step) % (unsigned)whole);
  auto block_of = [&](int t) __attribute__((always_inline)) {
    if (tail_first && t == 0) return whole;
    const int x = t - (tail_first ? 1 : 0) + rotated;
    return x < whole ? x : x - whole;
  };
  uint32_t off[T::DIRECT ? T::LOADS : 1];
  if constexpr (T::DIRECT) {
#pragma unroll
    for (int v = 0; v < T::LOADS; ++v) {
      int row, chunk;
      slot(v, lane, row, chunk);
      off[v] = (uint32_t)(v < T::A_LOADS ? a_row(row) * c.lda : (int64_t)b_row(row) * c.ldb) +
               16 * chunk;
    }
  }
  auto copy = [&](int t, int v) __attribute__((always_inline)) {
    const int8_t* base = (v < T::A_LOADS ? a_tile : b_tile) + block_of(t) * kBlockK;
    if (T::ONCE && v >= T::A_LOADS)
      dma16_sbase_once(base, off[v], lds_base + slot_at(v, t));
    else
      dma16_sbase_u(base, off[v], lds_base + slot_at(v, t));
  };
  // K tile t through registers, any alignment: loaded, and later stored.
  u32x4 held[T::LOADS];
  auto load_tile = [&](int t) __attribute__((always_inline)) {
    const int k0 = block_of(t) * kBlockK;
    const bool cut = T::DIRECT || k0 + kBlockK > c.K;
#pragma unroll
    for (int v = 0; v < T::LOADS; ++v) {
      int row, chunk;
      slot(v, lane, row, chunk);
      const int8_t* at = v < T::A_LOADS ? a_tile + a_row(row) * c.lda
                                        : b_tile + (int64_t)b_row(row) * c.ldb;
      const int k = k0 + 16 * chunk;
      held[v] = cut ? load16_row(at, k, c.K) : load16(at + k);
    }
  };
  auto store_tile = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < T::LOADS; ++v)
      *reinterpret_cast<u32x4*>(lds + slot_at(v, t) + 16 * lane) = held[v];
  };

  // The scales and bias that the epilogue will need, one row of the tile a thread.
  static_assert(T::THREADS >= T::BM && T::THREADS >= T::BN, "a thread for every row");
  float sa = 0.0f, sb = 0.0f, bias = 0.0f;
  if ((int)threadIdx.x < T::BN) {
    const int64_t n = group_b + n0 + b_row(threadIdx.x);
    if (c.K != 0) sb = c.SB[n];
    if (c.bias != nullptr) bias = c.bias[n];
  }
  if ((int)threadIdx.x < T::BM && c.K != 0)
    sa = c.SA[a_row(threadIdx.x) + (c.index != nullptr ? 0 : m0)];

  i32x16 sum[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) sum[i][j] = i32x16{};

  // This lane's chunk of a fragment row in step s is (2 s + half) permuted.
  const uint32_t swizzled = 16 * (half ^ ((l32 >> 1) & 7));
  const uint32_t a_frag = (wm * T::WTM + l32) * kBlockK;
  const uint32_t b_frag = T::B_AT + (wn * T::WTN + l32) * kBlockK;
  auto read_a = [&](I8Frags<T>& f, int t, int s, int blocks = T::FM) __attribute__((always_inline)) {
    const uint8_t* st = lds + t % T::STAGES * T::A_BYTES + (swizzled ^ (32 * s)) + a_frag;
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
      if (i < blocks) f.a[i] = *reinterpret_cast<const i32x4*>(st + i * 32 * kBlockK);
  };
  auto read_b = [&](I8Frags<T>& f, int t, int s) __attribute__((always_inline)) {
    const uint8_t* st = lds + (T::OWN_B ? 0 : t % T::STAGES * T::B_BYTES) + (swizzled ^ (32 * s)) + b_frag;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(st + j * 32 * kBlockK);
  };
  auto read = [&](I8Frags<T>& f, int t, int s) __attribute__((always_inline)) {
    read_a(f, t, s);
    read_b(f, t, s);
  };
  auto multiply = [&](const I8Frags<T>& f, int x) __attribute__((always_inline)) {
    const int i = x / T::FN, j = x % T::FN;
    sum[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[j], f.a[i], sum[i][j], 0, 0, 0);
  };
  I8Frags<T> f0, f1;

  // K tile t, whose first step's fragments are in f0; COPY: with the copies of tile t +
  // STAGES; MORE: tile t + 1 follows.
  constexpr int PRE = T::BLOCKS >= 4 ? 2 : 1;   // MFMAs that run while the waves meet
  auto k_tile = [&](int t, auto copy_next, auto more) __attribute__((always_inline)) {
    constexpr bool COPY = decltype(copy_next)::value, MORE = decltype(more)::value;
    read(f1, t, 1);
    if constexpr (!T::DIRECT && MORE) load_tile(t + 1);
#pragma unroll
    for (int x = 0; x < T::BLOCKS; ++x) multiply(f0, x);
    __builtin_amdgcn_sched_barrier(0);
    read(f0, t, 2);
#pragma unroll
    for (int x = 0; x < T::BLOCKS; ++x) multiply(f1, x);
    __builtin_amdgcn_sched_barrier(0);
    read(f1, t, 3);
#pragma unroll
    for (int x = 0; x < T::BLOCKS; ++x) multiply(f0, x);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!T::DIRECT && MORE) store_tile(t + 1);
#pragma unroll
    for (int x = 0; x < PRE; ++x) multiply(f1, x);
    if constexpr (MORE) {
      // Tile t + 1 has landed (younger copies may be on their way) and tile t is read.
      if constexpr (COPY)
        wait_vmcnt<(T::STAGES - 2) * T::LOADS>();
      else
        wait_vmcnt<0>();
      lds_barrier();
      read(f0, t + 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    // The copies between the last MFMAs (all at once would hold every wave at issue).
    constexpr int REST = T::BLOCKS - PRE;
#pragma unroll
    for (int x = 0; x < REST || (x == 0 && REST == 0); ++x) {
      if (x < REST) multiply(f1, PRE + x);
      if constexpr (COPY) {
        constexpr int OVER = REST > 0 ? REST : 1;
#pragma unroll
        for (int v = x * T::LOADS / OVER; v < (x + 1) * T::LOADS / OVER; ++v) copy(t + T::STAGES, v);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // The same for waves that own their rows of B: all of a K tile's fragments of B are
  // read at its start, then their one stage takes the next tile's; one meeting, at the
  // start.  PART: of the tile's rows of A only the first `live` blocks of 32 exist, as at the
  // end of a group; the others are neither copied nor multiplied (1024 tokens, 128 rows a
  // group on average, on 64 experts of 2048 x 4096 163 us without, 143 with).
  const int live = m_end - m0 >= T::BM ? T::FM : (m_end - m0 + 31) / 32;
  auto k_tile_own = [&](int t, auto copy_next, auto part) __attribute__((always_inline)) {
    constexpr bool COPY = decltype(copy_next)::value, PART = decltype(part)::value;
    wait_vmcnt<0>();
    lds_barrier();
    I8Frags<T> b1, b2, b3;   // (their fragments of B only)
    read_b(f0, t, 0);
    read_a(f0, t, 0, PART ? live : T::FM);
    read_b(b1, t, 1);
    read_b(b2, t, 2);
    read_b(b3, t, 3);
    // One step's products, with copies `first` .. `first` + `count` - 1 of the next tile between.
    auto step = [&](const I8Frags<T>& a, const I8Frags<T>& b, int first, int count)
        __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < T::BLOCKS; ++x) {
        const int i = x / T::FN, j = x % T::FN;
        if (!PART || i < live)
          sum[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b.b[j], a.a[i], sum[i][j], 0, 0, 0);
        if constexpr (COPY) {
#pragma unroll
          for (int v = first + x * count / T::BLOCKS; v < first + (x + 1) * count / T::BLOCKS; ++v) {
            __builtin_amdgcn_sched_barrier(0);
            if (!PART || v >= T::A_LOADS || (wave * T::A_LOADS + v) * 8 < 32 * live) copy(t + 1, v);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    read_a(f1, t, 1, PART ? live : T::FM);
    step(f0, f0, 0, T::A_LOADS);
    if constexpr (COPY) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);   // this wave's fragments of B are read
    }
    read_a(f0, t, 2, PART ? live : T::FM);
    step(f1, b1, T::A_LOADS, T::B_LOADS / 2);
    read_a(f1, t, 3, PART ? live : T::FM);
    step(f0, b2, T::A_LOADS + T::B_LOADS / 2, T::B_LOADS - T::B_LOADS / 2);
    step(f1, b3, 0, 0);
  };

  if constexpr (T::OWN_B) {
    if (kts > 0) {
      if (tail_first) {
        load_tile(0);
        store_tile(0);
      } else {
#pragma unroll
        for (int v = 0; v < T::LOADS; ++v) copy(0, v);
      }
      int t = 0;
      if (!T::GROUPED || live == T::FM) {
        for (; t + 1 < kts; ++t) k_tile_own(t, std::true_type(), std::false_type());
        k_tile_own(t, std::false_type(), std::false_type());
      } else if constexpr (T::GROUPED) {
        for (; t + 1 < kts; ++t) k_tile_own(t, std::true_type(), std::true_type());
        k_tile_own(t, std::false_type(), std::true_type());
      }
    }
  } else if (kts > 0) {
    if constexpr (T::DIRECT) {
#pragma unroll
      for (int first = 0; first < T::STAGES; ++first) {
        if (first >= kts) break;
        if (first == 0 && tail_first) {
          load_tile(0);
          store_tile(0);
        } else {
#pragma unroll
          for (int v = 0; v < T::LOADS; ++v) copy(first, v);
        }
      }
      if (kts >= T::STAGES)
        wait_vmcnt<(T::STAGES - 1) * T::LOADS>();
      else
        wait_vmcnt<0>();
    } else {
      load_tile(0);
      store_tile(0);
    }
    lds_barrier();
    read(f0, 0, 0);
    int t = 0;
    if constexpr (T::DIRECT)
      for (; t + T::STAGES < kts; ++t) k_tile(t, std::true_type(), std::true_type());
    for (; t + 1 < kts; ++t) k_tile(t, std::false_type(), std::true_type());
    k_tile(t, std::false_type(), std::false_type());
  }

  lds_barrier();   // every wave is done reading the stages
  {
    float* mb = reinterpret_cast<float*>(lds + T::SCALES_AT);
    float* ma = mb + 3 * T::BN;
    const int x = threadIdx.x;
    if (x < T::BN) {
      const SplitScale s(sb);
      mb[x] = s.m;
      reinterpret_cast<int*>(mb)[T::BN + x] = s.e;
      mb[2 * T::BN + x] = bias;
    }
    if (x < T::BM) {
      const SplitScale s(sa, c.alpha_e);
      ma[x] = s.m;
      reinterpret_cast<int*>(ma)[T::BM + x] = s.e;
    }
  }
  lds_barrier();
  if (c.act == GEMM_ACT_NONE)
    i8_write_as<T, 0>(c, sum, lds, wave, m0, m_end, n0, lane);
  else if (c.act == GEMM_ACT_GELU_TANH)
    i8_write_as<T, 1>(c, sum, lds, wave, m0, m_end, n0, lane);
  else
    i8_write_as<T, 2>(c, sum, lds, wave, m0, m_end, n0, lane);
}

namespace {

template <int BM, int BN, int WM, int WN, int STAGES, bool DIRECT, bool OWN_B>
hipError_t launch_tile(const I8Call& c, bool once, hipStream_t s) {
  const int tiles_m = (int)i8_tiles_m(c, BM);
  const int tiles_n = (int)((i8_b_rows(c) + BN - 1) / BN);
  // Where the bytes of the weights bound the call (groups; few rows) different weights start at different K,
  // the tiles that share them at the same: 512 tokens on 64 experts of 2048 x 4096 138 us
  // without, 106 with; 64 rows by 28672 x 4096 31 and 27.  Many rows of one weight are 2 to 4 %
  // slower with it, since tiles side by side then read A at different times.
  const I8TileArgs p{c, tiles_m, tiles_n, c.groups > 0 ? 4 : 8, c.groups > 0 ? 11 : 0,
                     c.groups == 0 && c.M <= 256 ? 11 : 0};
  const dim3 grid((unsigned)tiles_m * tiles_n), block(WM * WN * kWave);
  once = once && DIRECT;
  if (c.groups > 0 && once)
    i8_tile_kernel<I8Tile<BM, BN, WM, WN, STAGES, DIRECT, OWN_B, true, DIRECT>><<<grid, block, 0, s>>>(p);
  else if (c.groups > 0)
    i8_tile_kernel<I8Tile<BM, BN, WM, WN, STAGES, DIRECT, OWN_B, true, false>><<<grid, block, 0, s>>>(p);
  else if (once)
    i8_tile_kernel<I8Tile<BM, BN, WM, WN, STAGES, DIRECT, OWN_B, false, DIRECT>><<<grid, block, 0, s>>>(p);
  else
    i8_tile_kernel<I8Tile<BM, BN, WM, WN, STAGES, DIRECT, OWN_B, false, false>><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

bool i8_direct(const I8Call& c) {
  // 32-bit byte offsets from a tile's first row (from A's where rows are read by index,
  // over both halves of B with a gate).
  const int64_t a_rows = c.index != nullptr ? c.a_rows : 256;
  const int64_t b_rows = 256 + (c.gated ? (int64_t)c.N : 0);
  return c.lda % 16 == 0 && c.ldb % 16 == 0 && (reinterpret_cast<uintptr_t>(c.A) & 15u) == 0 &&
         (reinterpret_cast<uintptr_t>(c.B) & 15u) == 0 && a_rows * c.lda < (1ll << 32) &&
         b_rows * c.ldb < (1ll << 32);
}

hipError_t launch_i8_tile(const I8Call& c, int tile, bool once, hipStream_t s) {
  switch (tile) {
    case 0: return launch_tile<256, 256, 2, 4, 2, true, false>(c, once, s);
    case 1: return launch_tile<128, 256, 1, 4, 2, true, true>(c, once, s);
    case 2: return launch_tile<128, 128, 2, 2, 2, true, false>(c, once, s);
    case 3: return launch_tile<64, 128, 2, 2, 3, true, false>(c, once, s);
    case 4: return launch_tile<64, 64, 2, 2, 4, true, false>(c, once, s);
    case 5: return launch_tile<32, 128, 1, 4, 4, true, false>(c, once, s);
    // (Eight waves, since each holds what it loads: 4096 x 4096 x 4095 127 us, with four 184, with
    // sixteen 163; 64 x 14336 x 4095 49, 79 and 43.)
    default: return launch_tile<128, 128, 2, 4, 2, false, false>(c, once, s);
  }
}

}  // namespace lasg
