// The block-scaled e4m3 product in output tiles staged through LDS (formula and
// the two ways to sum a block: fp8_kernels.hip), for outputs large enough that
// the matrix units bound it.
//
// One K tile is one block of 128 columns: rows of 128 bytes, copied from memory
// straight into LDS (16 bytes a lane, whole 128-byte lines) one to three tiles
// ahead.  Row r's eight 16-byte chunks lie permuted by (r / 2) % 8, so that the
// fragment reads of 16 neighbouring rows fall into 16 different bank groups.
// The block's scales travel the same way, 4 bytes a lane.
//
// A wave multiplies 32x32 blocks: over the 128 columns into a fresh sum (the
// 8-bit MFMA's first step starts from an inline zero), then sum x scale into the
// fp32 totals on the vector unit while the matrix unit works on the next
// block.  B is the first operand, so a lane holds the columns 8 q + 4 (lane / 32) + 0..3 of
// one row of C: one scale of A per lane and block, and 4-column stores.
//
// What bounds it: the scaling is 16 FMAs (64 cycles) of vector work beside 128
// cycles of 8-bit MFMAs in a block; with the operands widened, and a scale for
// every row of B, about 300 beside 256.  Two workgroups share a CU, so that one works
// while the other meets at its barrier or writes its results (a 256 x 256 tile of eight
// waves took 313 us); counted over the whole launch the vector unit is busy 54 % and
// the matrix unit 45 % of the time, waves wait 24 %, so neither alone is the bound.
// Measured, a pass among others, on the fastest of several cards (the slowest 5 % more): 4096 x 14336 x 4096 with GELU 256 us (1880 TFLOP/s; a
// plain 8-bit library product with one scale 185), the same with a scale for every row
// of B 331 (1450), with fp32 sums 456 to 468 (1030), with rows off 16-byte
// boundaries 1110 (433); 4096 x 4096 x 8192 with fp32 sums and a scale for every row of
// B 278 (990; vector 57 %, matrix 47 %; the library's bfloat16 rate is 1360).
#include <type_traits>

#include "dma_common.h"
#include "fp8_common.h"

namespace lasg {

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, bool FAST_, bool ROWB_,
          bool DIRECT_>
struct Fp8Tile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int STAGES = STAGES_;   // of LDS: K tiles that are multiplied or on their way
  static constexpr bool FAST = FAST_, ROWB = ROWB_;
  // Copies straight into LDS (rows of A and B on 16-byte boundaries, 32-bit
  // offsets), else through registers.
  static constexpr bool DIRECT = DIRECT_;
  static constexpr int WAVES = WAVES_M * WAVES_N, THREADS = WAVES * kWave;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  // Waves side by side only: each copies and reads its own rows of B, so one
  // stage of B is enough (refilled once the wave holds its fragments).
  static constexpr bool OWN_B = WAVES_M == 1;
  static constexpr int A_BYTES = BM * kBlockK, B_BYTES = BN * kBlockK;
  static constexpr int B_AT = STAGES * A_BYTES;
  // Scales, per stage BN, then BM floats.
  static constexpr int SCALES_AT = B_AT + (OWN_B ? 1 : STAGES) * B_BYTES;
  static constexpr int SCALE_BYTES = 4 * (BM + BN);
  static constexpr int LDS_BYTES = SCALES_AT + STAGES * SCALE_BYTES;
  static constexpr int A_LOADS = BM / 8 / WAVES, B_LOADS = BN / 8 / WAVES;   // per wave, 1 KiB each
  static constexpr int LOADS = A_LOADS + B_LOADS;
  static constexpr int SCALE_COPIES = (BM / 64 + BN / 64 + WAVES - 1) / WAVES;   // per wave
  static constexpr int PER_TILE = LOADS + SCALE_COPIES;   // copies of a K tile, per wave
  static constexpr int AHEAD = STAGES - 1;   // how far the copies run before the products
  static_assert(STAGES == 2 || (STAGES > 2 && DIRECT && !OWN_B), "stages");
  static_assert(AHEAD * PER_TILE <= 63, "copies on their way must fit vmcnt");
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "copies split evenly over waves");
  static_assert(WTM % 32 == 0 && WTN % 32 == 0 && (ROWB || 128 % WTN == 0), "wave tile");
  static_assert(LDS_BYTES * (STAGES == 2 ? 8 / WAVES : 1) <= 160 * 1024, "LDS");
};

struct Fp8TileArgs {
  Fp8Call c;
  int tiles_m, tiles_n, group_m;
};

namespace {

// Row (of the tile) and chunk that lane `lane` copies in load v of wave `wave`.
template <class T>
__device__ __forceinline__ void copy_slot(int v, int wave, int lane, int& row, int& chunk) {
  const bool b = v >= T::A_LOADS;
  const int idx = b ? wave * T::B_LOADS + v - T::A_LOADS : wave * T::A_LOADS + v;
  row = 8 * idx + lane / 8;
  chunk = (lane % 8) ^ ((row >> 1) & 7);
}

// Where it puts them, in the stage of K tile number t.
template <class T>
__device__ __forceinline__ uint32_t copy_lds(int v, int wave, int t) {
  return v < T::A_LOADS ? t % T::STAGES * T::A_BYTES + (wave * T::A_LOADS + v) * 1024
                        : T::B_AT + (T::OWN_B ? 0 : t % T::STAGES * T::B_BYTES) +
                              (wave * T::B_LOADS + v - T::A_LOADS) * 1024;
}

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ const float* uniform(const float* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return reinterpret_cast<const float*>(lo | (uint64_t)hi << 32);
}

template <bool FAST>
struct Operand;   // 32 rows x 128 columns as the MFMAs take them
template <>
struct Operand<true> {
  i32x8 v[2];
  __device__ __forceinline__ void set(int s, u32x4 lo, u32x4 hi) {
    v[s] = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }
  static __device__ __forceinline__ f32x16 product(const Operand& b, const Operand& a) {
    f32x16 acc = {};
#pragma unroll
    for (int s = 0; s < 2; ++s)
      acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.v[s], a.v[s], acc, 0, 0, 0, 0, 0, 0);
    return acc;
  }
};
template <>
struct Operand<false> {
  bf16x8 v[2][4];
  __device__ __forceinline__ void set(int s, u32x4 lo, u32x4 hi) {
    v[s][0] = widen_bf16(lo[0], lo[1]);
    v[s][1] = widen_bf16(lo[2], lo[3]);
    v[s][2] = widen_bf16(hi[0], hi[1]);
    v[s][3] = widen_bf16(hi[2], hi[3]);
  }
  static __device__ __forceinline__ f32x16 product(const Operand& b, const Operand& a) {
    f32x16 acc = {};
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[s][x], a.v[s][x], acc, 0, 0, 0);
    return acc;
  }
};

// total += sum x scale, with one scale per row of B (`sb`: this lane's columns)
// times it where there is one.
template <class T>
__device__ __forceinline__ void add(f32x16& total, const f32x16& sum, float scale, const float* sb) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f32x4 s4 = {scale, scale, scale, scale};
    if constexpr (T::ROWB) s4 = scale * *reinterpret_cast<const f32x4*>(sb + 8 * q);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      total[4 * q + e] = __builtin_fmaf(sum[4 * q + e], s4[e], total[4 * q + e]);
  }
}

// The results of a wave, 32 rows at a time: bias and activation in registers,
// rounded to C's type, through the wave's own piece of LDS (chunks permuted as
// above) so that whole rows of 64 to 256 bytes are stored, 16 bytes a
// lane.  The activation and the width of C are chosen outside the loops.
template <class T, int ACT, bool WIDE>
__device__ __forceinline__ void write_back(const Fp8Call& c, const f32x16 (&total)[T::FM][T::FN],
                                           uint8_t* region, int m0, int n0, int wm, int wn,
                                           int lane) {
  constexpr int SIZE = WIDE ? 4 : 2, ROW = T::WTN * SIZE, CHUNKS = ROW / 16;
  constexpr int LINE = ROW >= 256 ? 1 : 256 / ROW;   // rows in a line of the LDS banks
  static_assert(1024 % ROW == 0, "whole rows per store");
  const int l32 = lane % 32, half = lane / 32;
  const int col0 = n0 + wn * T::WTN;
  const bool f16 = c.type == GEMM_TYPE_F16;
  f32x4 bias[T::FN][4];
#pragma unroll
  for (int j = 0; j < T::FN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = col0 + 32 * j + 8 * q + 4 * half;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        bias[j][q][e] = c.bias != nullptr && col + e < c.N ? c.bias[col + e] : 0.0f;
    }
  auto slot = [](int row, int chunk) {
    return row * ROW + 16 * (chunk ^ (row / LINE & (CHUNKS - 1)));
  };
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = apply_act(__builtin_fmaf(c.alpha, total[i][j][4 * q + e], bias[j][q][e]), ACT);
        if constexpr (WIDE) {
          *reinterpret_cast<f32x4*>(region + slot(l32, 8 * j + 2 * q + half)) = v;
        } else {
          uint16_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = f16 ? LmF16::bits(v[e]) : LmBF16::bits(v[e]);
          *reinterpret_cast<u32x2*>(region + slot(l32, 4 * j + q) + 8 * half) =
              __builtin_bit_cast(u32x2, h);
        }
      }
    asm volatile("" ::: "memory");   // (one wave's LDS accesses keep their order)
#pragma unroll
    for (int it = 0; it < 32 * ROW / 1024; ++it) {
      const int r = it * (1024 / ROW) + lane / CHUNKS, chunk = lane % CHUNKS;
      const u32x4 v = *reinterpret_cast<const u32x4*>(region + slot(r, chunk));
      const int row = m0 + wm * T::WTM + 32 * i + r, col = col0 + chunk * (16 / SIZE);
      if (row >= c.M || col >= c.N) continue;
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

}  // namespace

template <class T>
__global__ void __launch_bounds__(T::THREADS) __attribute__((amdgpu_waves_per_eu(2)))
fp8_tile_kernel(Fp8TileArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS_BYTES];
  const Fp8Call& c = p.c;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const int l32 = lane % 32, half = lane / 32;
  const uint32_t lds_base = lds_offset(lds);
  int tile_m, tile_n;
  tile_of_workgroup(blockIdx.x, p.tiles_m, p.tiles_n, p.group_m, tile_m, tile_n);
  const int m0 = tile_m * T::BM, n0 = tile_n * T::BN;
  const uint8_t* a_tile = c.A + (int64_t)m0 * c.lda;
  const uint8_t* b_tile = c.B + (int64_t)n0 * c.ldb;
  const int kbs = (c.K + kBlockK - 1) / kBlockK;

  // Scales in pieces of 64, B's first (with waves side by side its own to each
  // wave), then A's; a wave past the last piece copies that again, so that
  // all waves have the same number of copies on their way.
  auto scale_piece = [&](int u) __attribute__((always_inline)) {
    constexpr int PIECES = T::BM / 64 + T::BN / 64;
    return wave + u * T::WAVES < PIECES ? wave + u * T::WAVES : PIECES - 1;
  };
  const float* scales[T::SCALE_COPIES];
  int64_t scale_ld[T::SCALE_COPIES];
  uint32_t scale_off[T::SCALE_COPIES];
#pragma unroll
  for (int u = 0; u < T::SCALE_COPIES; ++u) {
    const int piece = scale_piece(u);
    const bool b = piece < T::BN / 64;
    const int row = 64 * (b ? piece : piece - T::BN / 64) + lane;
    const int last = b ? c.N - 1 - n0 : c.M - 1 - m0, at = row < last ? row : last;
    scales[u] = b ? c.SB + (T::ROWB ? n0 : n0 / kBlockK) : c.SA + m0;
    scale_ld[u] = b ? c.ldsb : c.ldsa;
    scale_off[u] = 4 * (b && !T::ROWB ? (n0 + at) / kBlockK - n0 / kBlockK : at);
  }

  // K tiles in the order they are taken.  A last, shorter block of K goes
  // through registers, with zeros behind it; where whole blocks are copied
  // straight into LDS it is taken first, so that its latency falls together
  // with the first copies'.
  const bool tail_first = T::DIRECT && c.K % kBlockK != 0;
  auto block_of = [&](int t) __attribute__((always_inline)) {
    return !tail_first ? t : t == 0 ? kbs - 1 : t - 1;
  };
  // (`l`: the lane.  Rows past the end read the last; 24 bits hold a row of the tile
  // and, with 256 rows within 2^31 bytes, a leading dimension.)
  auto copy = [&](int t, int v, int l) __attribute__((always_inline)) {
    int row, chunk;
    copy_slot<T>(v, wave, l, row, chunk);
    const bool b = v >= T::A_LOADS;
    const int last = b ? c.N - 1 - n0 : c.M - 1 - m0;
    dma16_sbase_u((b ? b_tile : a_tile) + block_of(t) * kBlockK,
                  __umul24(row < last ? row : last, b ? c.ldb : c.lda) + 16 * chunk,
                  lds_base + copy_lds<T>(v, wave, t));
  };
  auto copy_scales = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < T::SCALE_COPIES; ++u)
      dma4_sbase(uniform(scales[u] + block_of(t) * scale_ld[u]), scale_off[u],
                 __builtin_amdgcn_readfirstlane(lds_base + T::SCALES_AT +
                                                t % T::STAGES * T::SCALE_BYTES +
                                                256 * scale_piece(u)));
  };
  auto copy_by_hand = [&](int t, int l) __attribute__((always_inline)) {
    constexpr int BATCH = T::LOADS % 4 == 0 ? 4 : 2;
    static_assert(T::LOADS % BATCH == 0, "whole batches");
#pragma unroll 1
    for (int v0 = 0; v0 < T::LOADS; v0 += BATCH) {
      u32x4 x[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        int row, chunk;
        copy_slot<T>(v0 + u, wave, l, row, chunk);
        const bool b = v0 + u >= T::A_LOADS;
        const int last = b ? c.N - 1 - n0 : c.M - 1 - m0;
        x[u] = load16_row((b ? b_tile : a_tile) +
                              (int64_t)(row < last ? row : last) * (b ? c.ldb : c.lda),
                          block_of(t) * kBlockK + 16 * chunk, c.K);
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        *reinterpret_cast<u32x4*>(lds + copy_lds<T>(v0 + u, wave, t) + 16 * l) = x[u];
    }
  };

  f32x16 total[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) total[i][j] = f32x16{};

  constexpr int BLOCKS = T::FM * T::FN;
  f32x16 sum[2] = {{}, {}};
  float scale[2] = {0.0f, 0.0f};
  static_assert(BLOCKS % 2 == 0 || BLOCKS == 1, "sums alternate over K tiles too");
  constexpr bool LATE = !T::ROWB && BLOCKS > 1;   // a K tile's last block waits for the next tile

  // This lane's fragment chunks: (s, x) = k step, 16-byte half of the 32 bytes.
  const int swizzled = 16 * ((2 * half) ^ ((l32 >> 1) & 7));
  const uint32_t frag = l32 * kBlockK;

  // K tile t; COPY: with the direct copies of tile t + AHEAD.
  auto k_tile = [&](int t, auto copy_next) __attribute__((always_inline)) {
    constexpr bool COPY = decltype(copy_next)::value;
    int l = lane;
    // Where the registers are full the copies' offsets are formed anew each time
    // (held over the loop they would take those of a sum).
    if constexpr (T::OWN_B || !T::DIRECT) asm volatile("" : "+v"(l));
    // Tile t has landed (younger copies may be on their way), and every wave is
    // done with tile t - 1, whose stage takes tile t + AHEAD.
    constexpr int AHEAD = T::AHEAD;
    if constexpr (COPY)
      wait_vmcnt<(AHEAD - 1) * T::PER_TILE>();
    else
      wait_vmcnt<0>();
    lds_barrier();
    const uint8_t* a_st = lds + t % T::STAGES * T::A_BYTES + wm * T::WTM * kBlockK + frag;
    const uint8_t* b_st = lds + T::B_AT + (T::OWN_B ? 0 : t % T::STAGES * T::B_BYTES) +
                          wn * T::WTN * kBlockK + frag;
    const float* sb_st = reinterpret_cast<const float*>(lds + T::SCALES_AT +
                                                        t % T::STAGES * T::SCALE_BYTES) + wn * T::WTN;
    const float* sa_st = sb_st - wn * T::WTN + T::BN + wm * T::WTM + l32;
    auto read = [&](const uint8_t* base) {
      Operand<T::FAST> o;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        o.set(s, *reinterpret_cast<const u32x4*>(base + (swizzled ^ (64 * s))),
              *reinterpret_cast<const u32x4*>(base + (swizzled ^ (64 * s) ^ 16)));
      return o;
    };
    Operand<T::FAST> a, b[T::FN];
#pragma unroll
    for (int j = 0; j < T::FN; ++j) b[j] = read(b_st + j * 32 * kBlockK);
    const float sb0 = T::ROWB ? 1.0f : sb_st[0];
    float sa[T::FM];
#pragma unroll
    for (int i = 0; i < T::FM; ++i) sa[i] = sa_st[32 * i];
    a = read(a_st);
    // Block x's matrix instructions go out before block x - 1's sum is scaled,
    // so that the vector unit works under them; the last block of a K tile is
    // scaled in the next one, under the latency of its first reads.
#pragma unroll
    for (int x = 0; x < BLOCKS; ++x) {
      const int i = x / T::FN, j = x % T::FN;
      if (!T::DIRECT && j == 0 && i > 0) a = read(a_st + i * 32 * kBlockK);
      if (x == 0 && LATE) {
        add<T>(total[T::FM - 1][T::FN - 1], sum[1], scale[1], nullptr);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (x == 0 && COPY) copy_scales(t + AHEAD);
      sum[x & 1] = Operand<T::FAST>::product(b[j], a);
      scale[x & 1] = sa[i] * sb0;
      if (T::DIRECT && j == T::FN - 1 && i + 1 < T::FM) a = read(a_st + (i + 1) * 32 * kBlockK);
      __builtin_amdgcn_sched_barrier(0);
      // The next tile's copies, some under each block's matrix instructions (all
      // at once would hold every wave at issue for about a thousand cycles), the
      // last well before the tile's end.  By block FN - 1 a wave has read its
      // fragments of B.
      if constexpr (COPY) {
        constexpr int FIRST = T::OWN_B ? T::FN - 1 : 0;
        constexpr int OVER = BLOCKS > 4 ? BLOCKS / 2 : BLOCKS - FIRST;
        if (x >= FIRST && x < FIRST + OVER) {
#pragma unroll
          for (int v = (x - FIRST) * T::LOADS / OVER; v < (x - FIRST + 1) * T::LOADS / OVER; ++v)
            copy(t + AHEAD, v, l);
        }
      }
      if (x > 0) {
        const int pi = (x - 1) / T::FN, pj = (x - 1) % T::FN;
        add<T>(total[pi][pj], sum[(x - 1) & 1], scale[(x - 1) & 1], sb_st + 32 * pj + 4 * half);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (!LATE)   // (scales per row of B lie in the stage)
      add<T>(total[T::FM - 1][T::FN - 1], sum[(BLOCKS - 1) & 1], scale[(BLOCKS - 1) & 1],
             sb_st + 32 * (T::FN - 1) + 4 * half);
    if (!T::DIRECT && t + 1 < kbs) {
      copy_scales(t + 1);
      asm volatile("" : "+v"(l));
      copy_by_hand(t + 1, l);
    }
  };
#pragma unroll
  for (int first = 0; first < T::AHEAD; ++first) {
    if (first >= kbs) break;
    copy_scales(first);
    if (T::DIRECT && !(first == 0 && tail_first)) {
#pragma unroll
      for (int v = 0; v < T::LOADS; ++v) copy(first, v, lane);
    } else {
      copy_by_hand(first, lane);
    }
  }
  int t = 0;
  if constexpr (T::DIRECT)
    for (; t + T::AHEAD < kbs; ++t) k_tile(t, std::true_type());
  for (; t < kbs; ++t) k_tile(t, std::false_type());
  if constexpr (LATE) add<T>(total[T::FM - 1][T::FN - 1], sum[1], scale[1], nullptr);

  lds_barrier();   // every wave is done reading the stages
  static_assert(T::WAVES * 32 * T::WTN * 4 <= T::LDS_BYTES, "staging of 32 rows a wave");
  uint8_t* region = lds + wave * (32 * T::WTN * 4);
  const bool wide = c.type == GEMM_TYPE_F32;
  if (c.act == GEMM_ACT_NONE)
    wide ? write_back<T, 0, true>(c, total, region, m0, n0, wm, wn, lane)
         : write_back<T, 0, false>(c, total, region, m0, n0, wm, wn, lane);
  else if (c.act == GEMM_ACT_GELU_TANH)
    wide ? write_back<T, 1, true>(c, total, region, m0, n0, wm, wn, lane)
         : write_back<T, 1, false>(c, total, region, m0, n0, wm, wn, lane);
  else
    wide ? write_back<T, 2, true>(c, total, region, m0, n0, wm, wn, lane)
         : write_back<T, 2, false>(c, total, region, m0, n0, wm, wn, lane);
}

namespace {

template <class T>
hipError_t launch_tile(const Fp8Call& c, hipStream_t s) {
  const Fp8TileArgs p{c, (c.M + T::BM - 1) / T::BM, (c.N + T::BN - 1) / T::BN, 8};
  fp8_tile_kernel<T><<<dim3((unsigned)p.tiles_m * p.tiles_n), T::THREADS, 0, s>>>(p);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int STAGES, bool DIRECT>
hipError_t launch_as(const Fp8Call& c, hipStream_t s) {
  if (c.fast_sums)
    return c.b_rows == 1 ? launch_tile<Fp8Tile<BM, BN, WM, WN, STAGES, true, true, DIRECT>>(c, s)
                         : launch_tile<Fp8Tile<BM, BN, WM, WN, STAGES, true, false, DIRECT>>(c, s);
  return c.b_rows == 1 ? launch_tile<Fp8Tile<BM, BN, WM, WN, STAGES, false, true, DIRECT>>(c, s)
                       : launch_tile<Fp8Tile<BM, BN, WM, WN, STAGES, false, false, DIRECT>>(c, s);
}

}  // namespace

bool fp8_direct(const Fp8Call& c) {
  return c.lda % 16 == 0 && c.ldb % 16 == 0 && (reinterpret_cast<uintptr_t>(c.A) & 15u) == 0 &&
         (reinterpret_cast<uintptr_t>(c.B) & 15u) == 0 &&
         c.lda < (1 << 23) && c.ldb < (1 << 23);   // 256 rows within 2^31 bytes, 24-bit products
}

hipError_t launch_fp8_tile(const Fp8Call& c, int tile, hipStream_t s) {
  switch (tile) {
    case 0: return launch_tile<Fp8Tile<128, 256, 1, 4, 2, true, false, true>>(c, s);
    case 1: return launch_as<128, 128, 2, 2, 2, true>(c, s);
    case 2: return launch_as<64, 64, 2, 2, 4, true>(c, s);
    case 3: return launch_as<64, 64, 2, 2, 3, true>(c, s);   // (three workgroups per CU)
    default: return launch_as<128, 128, 2, 2, 2, false>(c, s);
  }
}

}  // namespace lasg
