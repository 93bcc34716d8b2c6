// What the two kernel files of the int8 product share.
#pragma once

#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// The tiled kernels (i8_tile_kernels.hip): tiles 0 to 6 of i8_tile.  Tiles 0 to 5
// copy straight into LDS, which the call has to allow (i8_direct); `once`: B past the caches.
bool i8_direct(const I8Call& c);
hipError_t launch_i8_tile(const I8Call& c, int tile, bool once, hipStream_t s);

// Rows of B, of a group where there are groups.
__host__ __device__ __forceinline__ int64_t i8_b_rows(const I8Call& c) {
  return (int64_t)c.N << c.gated;
}
// Tiles of `bm` rows that a call can have: with groups every one may end inside a tile.
__host__ __device__ __forceinline__ int64_t i8_tiles_m(const I8Call& c, int bm) {
  const int64_t whole = ((int64_t)c.M + bm - 1) / bm;
  if (c.groups == 0) return whole;
  const int64_t most = (int64_t)c.M / bm + (c.groups < c.M ? c.groups : c.M);
  return most > whole ? most : whole;
}

// A scale as mantissa and exponent, so that the product of a sum, its two scales and
// alpha (I8Call) neither underflows nor overflows before it is whole: the exponents of all three are
// added first (alpha's to the row's), and alpha's mantissa, at least 1, comes last, in one fma with the bias.
struct SplitScale {
  float m;
  int e;
  __device__ __forceinline__ explicit SplitScale(float s, int more = 0)
      : m(__builtin_amdgcn_frexp_mantf(s)), e(__builtin_amdgcn_frexp_expf(s) + more) {}
};
// alpha sa sb sum + bias (ea with alpha's exponent): the sum is exact and is rounded to fp32 here, once.
__device__ __forceinline__ float i8_scaled(int sum, float ma, int ea, float mb, int eb, float alpha,
                                           float bias) {
  return __builtin_fmaf(alpha, __builtin_ldexpf((float)sum * (ma * mb), ea + eb), bias);
}

// A group's rows, kept inside 0 .. M whatever the offsets hold.
__device__ __forceinline__ void group_rows(const I8Call& c, int g, int& begin, int& end) {
  const int b = c.offsets[g], e = c.offsets[g + 1];
  begin = b < 0 ? 0 : b < c.M ? b : c.M;
  end = e < begin ? begin : e < c.M ? e : c.M;
}

// Tiles of BM rows that `rows` >= 0 take.  (Unsigned: of up to 2^31 - 1 rows the sum passes int.)
template <int BM>
__device__ __forceinline__ int tiles_of(int rows) {
  return (int)(((unsigned)rows + BM - 1) / BM);
}

// The tiles of BM rows of all groups, in order: their number, and tile t's
// group and rows.  A wave works it out alone: lane l looks after the groups l, ...
// of `per` consecutive ones, whose tiles are summed over the lanes.
template <int BM>
struct GroupTiles {
  int total;     // in every lane, scalar
  int per, sum, mine;
  __device__ __forceinline__ explicit GroupTiles(const I8Call& c) {
    const int lane = threadIdx.x % kWave;
    per = (c.groups + kWave - 1) / kWave;
    mine = 0;
    for (int x = 0; x < per; ++x) {
      const int g = lane * per + x;
      if (g < c.groups) {
        int b, e;
        group_rows(c, g, b, e);
        mine += tiles_of<BM>(e - b);
      }
    }
    sum = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const int y = __shfl_up(sum, d);
      if (lane >= d) sum += y;
    }
    // (Offsets that do not ascend may add up to more than the call was launched for, or past 2^31.)
    const int all = __builtin_amdgcn_readlane(sum, kWave - 1), most = (int)i8_tiles_m(c, BM);
    total = all < 0 ? 0 : all < most ? all : most;
  }
  // 0 <= t < total.  Of offsets that do not ascend a tile may come out empty (row >=
  // end), but never outside 0 .. M.
  __device__ __forceinline__ void find(const I8Call& c, int t, int& group, int& row, int& end) const {
    const uint64_t past = __ballot(sum > t);
    const int lane = past != 0 ? __builtin_ctzll(past) : 0;
    int left = t - __builtin_amdgcn_readlane(sum - mine, lane);
    group = lane * per;
    const int last = group + per < c.groups ? group + per - 1 : c.groups - 1;
    int b, e;
    group_rows(c, group, b, e);
    while (left >= tiles_of<BM>(e - b) && group < last) {
      left -= tiles_of<BM>(e - b);
      group_rows(c, ++group, b, e);
    }
    const bool good = left >= 0 && left < tiles_of<BM>(e - b);
    group = __builtin_amdgcn_readfirstlane(group);
    row = __builtin_amdgcn_readfirstlane(good ? b + left * BM : e);
    end = __builtin_amdgcn_readfirstlane(e);
  }
};

// The row of A that row r of the product reads.
__device__ __forceinline__ int64_t i8_a_row(const I8Call& c, int r) {
  if (c.index == nullptr) return r;
  const int i = c.index[r];
  const unsigned a = (unsigned)(i < 0 ? 0 : i) / (unsigned)c.per;
  return a < (unsigned)c.a_rows ? a : c.a_rows - 1;
}

}  // namespace lasg
