// block_scale.cuh -- scales of an e4m3 cache by block: one for the K and one for
// the V of each tile (16 tokens of a kv head).
//
// A scale is a power of two, held as its E8M0 byte (exponent + 127).  e4m3 is a
// floating-point format: a finer scale would gain no digit, only up to one
// binade of range, and with powers of two the product with 1 / scale is exact
// and codes that move to a larger scale keep their digits (only what falls below
// the smallest normal code, 2^-6, is rounded again).  Exponents lie within
// [kExpLow, kExpHigh], values within 448 2^30 = 4.8e11 and steps of 2^-59 for
// blocks of all but nothing; bytes outside count as the nearest bound, so that
// no byte makes an infinity, a NaN or a subnormal factor, and ratios of scales
// (at most 2^80) stay far inside fp32.
#pragma once

#include "common.cuh"

namespace fpk {

constexpr int kExpLow = -50, kExpHigh = 30;

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((127 + e) << 23); }

// The least exponent e with top <= 448 2^e, within the range (top >= 0, finite): 448 = 1.75 2^8.
__device__ __forceinline__ int block_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kExpLow), kExpHigh);
}

// The exponent that a byte stands for.
__device__ __forceinline__ int scale_exponent(uint32_t byte) {
  return min(max(static_cast<int>(byte) - 127, kExpLow), kExpHigh);
}

// |x| of a finite x, 0 of others.
__device__ __forceinline__ float finite_magnitude(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? __uint_as_float(u) : 0.f;
}

// Four e4m3 codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a.x * f, a.y * f), __NV_SATFINITE, __NV_E4M3)) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(b.x * f, b.y * f), __NV_SATFINITE, __NV_E4M3)) << 16;
}

// The first n (0 .. 16) of 16 codes times f, the others as they are.
__device__ __forceinline__ uint4 rescale_first(const uint4& x, int n, float f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = min(max(n - 4 * i, 0), 4);
    const uint32_t mine = k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
    y[i] = (rescale4(w[i], f) & mine) | (w[i] & ~mine);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

}  // namespace fpk
