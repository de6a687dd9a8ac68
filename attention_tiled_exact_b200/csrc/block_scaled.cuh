// The element format of the block-scaled 8-bit cache: E4M3 codes and one E8M0
// exponent byte for each (block, head).
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

namespace attn {
namespace bscale {

constexpr int BIAS = 127;
constexpr int E_MIN = -110, E_MAX = 120;  // exponents that the append writes

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The scale a byte stands for: 2^(byte - 127), 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  if (byte == 0) return __uint_as_float(0x00400000u);  // 2^-127, a subnormal
  return byte == 255 ? NAN : __uint_as_float(byte << 23);
}

// The smallest e of [E_MIN, E_MAX] with amax <= 448 * 2^e (448 = 1.75 * 2^8 is
// the largest E4M3 value), from amax's exponent and fraction bits.
__device__ __forceinline__ int exponent_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, E_MIN), E_MAX);
}

// Two E4M3 codes (low byte first) as an exact fp16 pair.
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t w) {
  uint32_t h2;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(w));
  return h2;
}

__device__ __forceinline__ float2 codes_to_float2(uint32_t w) {
  const uint32_t h2 = codes_to_f16x2(w);
  __half2 h;
  memcpy(&h, &h2, 4);
  return __half22float2(h);
}

// Eight codes as fp32 code values.
__device__ __forceinline__ void load_codes8(const uint8_t* p, float* x) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  const float2 a = codes_to_float2(r.x & 0xffffu), b = codes_to_float2(r.x >> 16);
  const float2 c = codes_to_float2(r.y & 0xffffu), d = codes_to_float2(r.y >> 16);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}

// Two fp32 values rounded to E4M3 (nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void store_codes8(uint8_t* p, const float* x, float mul) {
  uint2 r;
  r.x = to_codes(x[0] * mul, x[1] * mul) | (to_codes(x[2] * mul, x[3] * mul) << 16);
  r.y = to_codes(x[4] * mul, x[5] * mul) | (to_codes(x[6] * mul, x[7] * mul) << 16);
  *reinterpret_cast<uint2*>(p) = r;
}

}  // namespace bscale
}  // namespace attn
