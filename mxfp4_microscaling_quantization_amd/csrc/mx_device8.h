// Device-side building blocks of the 8-bit matrices (gfx950, wave64).
//
// An 8-bit matrix holds E4M3 codes (OCP: bit 7 sign, 4 exponent bits of bias 7, 3 mantissa bits,
// largest value 448, 0x7F and 0xFF NaN) and one E8M0 byte per 128 values, the smallest power of
// two 2^e with amax <= 448 2^e: 448 = 1.75 2^8, so e is the exponent of amax less 8, and one more
// where its mantissa is past 1.75.  No value is past the largest code, so nothing saturates.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

constexpr int kBlock8 = 128;

// Scale byte from the bit pattern of the block's largest magnitude: 0xFF for NaN or Inf, 0 (e =
// -127) at the lower end and for a block of zeros, at most 247.
__device__ __forceinline__ uint32_t scale8_byte_of(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  const uint32_t f = (amax + 0x1FFFFFu) >> 23;  // the carry of a mantissa past 1.75
  return f > 8u ? f - 8u : 0u;
}

// 2^e of a scale byte as a float32 factor of decoded codes (0xFF: NaN, whatever the code).
__device__ __forceinline__ float scale8_of(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : scale_of(byte);
}

// Largest pattern over the 16 lanes of a row.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = quad_max_u32(v);
  v = max(v, dpp_u32<0x124>(v));  // rotations by 4 and by 8 within the row
  v = max(v, dpp_u32<0x128>(v));
  return v;
}

// E4M3 codes of four values times inv = 2^-e: a value times a power of two is exact in float32
// but for results below 2^-126, which round to code 0 either way; the conversion rounds to
// nearest, ties to even, and keeps the sign of zeros.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

// The 8 codes of v under scale byte `byte` (0xFF: code 0).
__device__ __forceinline__ uint2 encode8(const float v[8], uint32_t byte) {
  if (byte == 255u) return make_uint2(0u, 0u);
  const float inv = inv_scale_of(byte);
  return make_uint2(encode4(v[0], v[1], v[2], v[3], inv), encode4(v[4], v[5], v[6], v[7], inv));
}

// Two float32 values as bf16, nearest even, a in the low half: one instruction (rounding by integer
// operations, as f32_to_bf16_rne, takes 15).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  const v2 r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// Exact values of 8 codes times a scale (values past the float32 range come out infinite).
__device__ __forceinline__ void decode8_e4m3(uint2 w, float scale, float v[8]) {
  const mx_v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false);
  const mx_v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
  const mx_v2f c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false);
  const mx_v2f d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
  v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
  v[4] = c.x * scale; v[5] = c.y * scale; v[6] = d.x * scale; v[7] = d.y * scale;
}

// 8 consecutive values of a row of cols from column col on, 0 from cols on.  T: float or uint16_t (bf16), at
// its own alignment.  Loads and conversion are apart, so that a thread's loads are all on their way before the
// first is waited for.  cols a multiple of 8 (ODD false): no branch, a run past the row loads its first columns;
// a branch around each load and its conversion made the next load wait.
template <typename T>
struct Run8 {
  T raw[8];
  template <bool ODD>
  __device__ __forceinline__ void load(const T* __restrict__ row, int64_t col, int64_t cols) {
    if constexpr (!ODD) {
      __builtin_memcpy(raw, row + (col < cols ? col : 0), sizeof(raw));
    } else if (cols >= 8) {  // the last run starts early, and its values are moved down
      __builtin_memcpy(raw, row + (col < cols - 8 ? col : cols - 8), sizeof(raw));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = row[col + i < cols ? col + i : 0];
    }
  }
  template <bool ODD>
  __device__ __forceinline__ void values(int64_t col, int64_t cols, bool there, float v[8]) const {
    const int64_t n = there ? cols - col : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = bf16_lo(raw[i]);
      else v[i] = raw[i];
    }
    if constexpr (ODD) {
      const int early = cols >= 8 && n < 8 ? (int)(8 - (n > 0 ? n : 0)) : 0;
#pragma unroll
      for (int d = 4; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = early & d ? (i + d < 8 ? v[i + d] : 0.0f) : v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (ODD ? i : 0) < n ? v[i] : 0.0f;
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, int64_t n, const float v[8]) {
  T raw[8];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = bf16_pair(v[2 * i], v[2 * i + 1]);
      __builtin_memcpy(raw + 2 * i, &w, 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = v[i];
  }
  if (n >= 8) {
    __builtin_memcpy(p, raw, sizeof(raw));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = raw[i];
  }
}

// Position of a thread in the flat order (row, lane of the row), `per` lanes a row: the
// workgroup's first index is divided in 64 bits once, the threads' in 32.
struct RowLane {
  int64_t row;
  int lane;
};
__device__ __forceinline__ RowLane row_lane(int64_t first, int at, int per) {
  const int64_t r0 = first / per;
  const uint32_t r = (uint32_t)(first - r0 * per) + (uint32_t)at;
  const uint32_t q = r / (uint32_t)per;
  return {r0 + q, (int)(r - q * (uint32_t)per)};
}

}  // namespace mx
