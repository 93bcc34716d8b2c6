// Device-side pieces shared by the 8-bit operators (block quantisation, the
// block-scaled product) and the mixture-of-experts layer: element types, loads
// at any byte alignment with zeros past the end, e4m3 conversion, activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"

namespace lasg {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The same vectors at any byte address: gfx950 serves global loads and stores
// of up to 16 bytes at any alignment, so rows of any length take the same code path.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

constexpr int kBlockK = 128;   // columns that share one scale

__device__ __forceinline__ u32x4 load16(const void* p) {
  return *static_cast<const u32x4_any*>(p);
}

// Bytes [at, at + 16) of a row of `bytes` bytes, zeros from its end on (at < 2^31 -
// 16; the row itself may start anywhere).  Nothing past the row is read: a chunk
// that crosses the end is the row's last 16 bytes, shifted; one wide load either
// way, and single bytes only in rows shorter than that.
__device__ __forceinline__ u32x4 load16_row(const void* row, int at, int bytes) {
  const uint8_t* p = static_cast<const uint8_t*>(row);
  if (bytes < 16) {
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int e = 0; e < 16 && at + e < bytes; ++e) {
      const uint32_t b = (uint32_t)p[at + e] << (8 * (e % 4));
      v[0] |= e / 4 == 0 ? b : 0u;
      v[1] |= e / 4 == 1 ? b : 0u;
      v[2] |= e / 4 == 2 ? b : 0u;
      v[3] |= e / 4 == 3 ? b : 0u;
    }
    return v;
  }
  const int from = at < bytes - 16 ? at : bytes - 16;
  const u32x4 v = load16(p + from);
  const int shift = 8 * (at - from < 16 ? at - from : 16);
  uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
  if (shift >= 64) {
    lo = shift < 128 ? hi >> (shift - 64) : 0;
    hi = 0;
  } else if (shift > 0) {
    lo = lo >> shift | hi << (64 - shift);
    hi >>= shift;
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
// Eight 16-bit elements at p of which the first `valid` (any number; <= 0 none)
// exist; the rest come back as zeros and are not read.
__device__ __forceinline__ u32x4 load8h_upto(const uint16_t* p, int valid) {
  if (valid >= 8) return load16(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < valid) v[e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
  return v;
}

// A value of an input array that is the same for the whole wave, through the
// scalar cache (a vector load for each scale took as many load instructions as the weights).
__device__ __forceinline__ float uniform_value(const float* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return *reinterpret_cast<const __attribute__((address_space(4))) float*>(lo | (uint64_t)hi << 32);
}

// Eight e4m3 bytes as eight 16-bit values.  Exact: e4m3's 4 significant bits
// and its exponents -9 .. 8 are normal numbers of bfloat16, and of binary16.
__device__ __forceinline__ bf16x8 widen_bf16(uint32_t lo, uint32_t hi) {
  bf16x2 v[4];
  v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f16x8 widen_f16(uint32_t lo, uint32_t hi) {
  f16x2 v[4];
  v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return __builtin_bit_cast(f16x8, v);
}

// The 16-bit formats with their 16x16x32 MFMA (lane l: eight k of row l % 16 of
// either operand; lane l of the result: column l % 16, rows 4 (l / 16) + 0..3).
struct LmF16 {
  typedef f16x8 vec8;
  static __device__ __forceinline__ f32x4 mfma(vec8 a, vec8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ vec8 widen(uint32_t lo, uint32_t hi) { return widen_f16(lo, hi); }
  static __device__ __forceinline__ uint16_t bits(float x) {
    return __builtin_bit_cast(uint16_t, (_Float16)x);
  }
  static __device__ __forceinline__ float value(uint16_t b) {
    return (float)__builtin_bit_cast(_Float16, b);
  }
  // Largest finite value: inner activations are clamped to it (see moe_kernels.hip).
  static constexpr float kMax = 65504.0f;
  static constexpr bool kNarrow = true;   // fewer exponents than fp32
};
struct LmBF16 {
  typedef bf16x8 vec8;
  static __device__ __forceinline__ f32x4 mfma(vec8 a, vec8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ vec8 widen(uint32_t lo, uint32_t hi) { return widen_bf16(lo, hi); }
  static __device__ __forceinline__ uint16_t bits(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
  }
  static __device__ __forceinline__ float value(uint16_t b) {
    return __builtin_bit_cast(float, (uint32_t)b << 16);
  }
  static constexpr float kMax = 3.3895313892515355e38f;
  static constexpr bool kNarrow = false;
};

// x times a factor: GELU in its tanh form is x / (1 + exp(-2u)) with u =
// sqrt(2/pi) (x + 0.044715 x^3), SiLU is x / (1 + exp(-x)).  The hardware
// base-2 exponential and reciprocal are within about an ulp of fp32.
// `act`: 0 identity, 1 GELU, 2 SiLU (uniform over the launch).
__device__ __forceinline__ float apply_act(float x, int act) {
  if (act == 0) return x;
  const float c = act == 1 ? -2.302208198f * __builtin_fmaf(0.044715f * x, x * x, x)
                           : -1.442695041f * x;
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(c));
}

}  // namespace lasg
