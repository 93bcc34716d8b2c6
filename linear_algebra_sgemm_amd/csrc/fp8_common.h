// What the kernels of the block-scaled product share: the store of a result.
#pragma once

#include "lm_common.h"
#include "lm_launch.h"

namespace lasg {

// Four consecutive values of one row of C (columns col ..; `left` of them exist).
__device__ __forceinline__ void store_c(const Fp8Call& p, int64_t row, int64_t col, f32x4 v) {
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

// The tiled kernels (fp8_tile_kernels.hip): tiles 0 to 4 of fp8_tile.  Tiles 0
// to 3 copy straight into LDS, which the call has to allow (fp8_direct).
bool fp8_direct(const Fp8Call& c);
hipError_t launch_fp8_tile(const Fp8Call& c, int tile, hipStream_t s);

}  // namespace lasg
