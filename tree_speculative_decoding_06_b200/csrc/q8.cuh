// The 8-bit cache format: e4m3 codes with one power-of-two scale byte per (block of tokens, KV head).
//
// value = code * 2^(byte - 127).  A power of two costs the format nothing (e4m3 is itself a floating
// point type) and buys three things: the value is exact in bf16, a block whose scale grows is
// requantised by an exponent shift, and the attention applies scales by adding exponents.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace tsd {
namespace q8 {

constexpr int kByteMin = 87;          // 2^-40: an all-zero block; also keeps the attention's P * 2^k normal
constexpr int kByteMax = 247;         // 2^120: the scale of the largest floats

// Byte of the smallest power of two 2^k, k >= -40, with amax <= 448 * 2^k (448 = 1.75 * 2^8), from the
// bits of amax (finite, >= 0): k = e - 8 when the significand is at most 1.75, else e - 7.
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23);                       // biased exponent; subnormals end at the floor below
  const int k = e - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return k < kByteMin ? kByteMin : k;
}
// 2^(byte - 127), byte in [1, 254].
__device__ __forceinline__ float pow2_byte(int byte) { return __uint_as_float((uint32_t)byte << 23); }
// 1 / 2^(byte - 127) (byte in [1, 253], so the result is normal).
__device__ __forceinline__ float inv_pow2_byte(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
// Bytes outside [1, 253] are never written; a reader clamps so that a stray one cannot make a NaN.
__device__ __forceinline__ int clean_byte(int byte) { return min(max(byte, 1), 253); }

// |x| where x is finite, else 0: infinities saturate and NaN stays NaN, neither sets the scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Two values to two codes, round to nearest even, saturating (NaN -> 0x7f); lo in the low byte.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return encode2(a, b) | (encode2(c, d) << 16);
}
// At the largest scale 256 * 2^120 is past the largest float: its codes (not NaN's) saturate at 240.
__device__ __forceinline__ uint32_t saturate240(uint32_t w) {
  const uint32_t m = w & 0x7f7f7f7fu, nan = __vcmpeq4(m, 0x7f7f7f7fu);
  return (w & 0x80808080u) | (m & nan) | (__vminu4(m, 0x77777777u) & ~nan);
}
// Two codes to two floats (exact).
__device__ __forceinline__ float2 decode2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}
// Four codes of a word to two bf16 pairs of code * scale (scale a power of two: exact).
__device__ __forceinline__ uint2 decode4_bf16(uint32_t w, float scale) {
  const float2 a = decode2(w), b = decode2(w >> 16);
  return make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale));
}

}  // namespace q8
}  // namespace tsd
