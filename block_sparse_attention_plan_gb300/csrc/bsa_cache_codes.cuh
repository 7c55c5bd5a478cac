// 8-bit codes of the cache (E4M3 and INT8): conversions between codes and
// fp32 / packed fp16.  Every code is exact in fp16 (E4M3 has 4 significant
// bits and exponents from 2^-9 to 2^8, the integers 7 bits).
#pragma once

#include <cstdint>

#include "bsa.h"

namespace bsa {
namespace dev {

// Largest code, and the exponent and fraction the scale rule compares with:
// 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6.
template <int KIND>
struct CodeRange {
  static constexpr float top = KIND == BSA_CACHE_INT8 ? 127.f : 448.f;
  static constexpr int exp = KIND == BSA_CACHE_INT8 ? 6 : 8;
  static constexpr uint32_t frac = KIND == BSA_CACHE_INT8 ? 0x7e0000u : 0x600000u;  // fp32 fraction bits of top
};
constexpr int kCacheMinExp = -100;

// Smallest 2^e, e >= kCacheMinExp, with amax <= top * 2^e (amax finite, >= 0):
// amax = (1 + f) 2^k needs e = k - exp(top), or one more where f exceeds top's
// fraction.  Integer arithmetic: no rounding decides it.
template <int KIND>
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 127 - CodeRange<KIND>::exp + ((b & 0x7fffffu) > CodeRange<KIND>::frac ? 1 : 0);
  e = e < kCacheMinExp ? kCacheMinExp : e;  // (zero and fp32 subnormals land here)
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two codes (low byte from `lo`), rounded to nearest even, saturated.
template <int KIND>
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  if constexpr (KIND == BSA_CACHE_INT8) {
    int a, b;  // cvt.rni.sat to s8: ties to even, -128 only from below -127.5; NaN gives 0
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(a) : "f"(fmaxf(lo, -127.f)));
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(b) : "f"(fmaxf(hi, -127.f)));
    if (lo != lo) a = 0;  // fmaxf drops a NaN
    if (hi != hi) b = 0;
    return ((uint32_t)a & 0xffu) | ((uint32_t)b & 0xffu) << 8;
  } else {
    uint16_t r;  // the first source becomes the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
}

// Packed fp16 of the codes in the low / high 16 bits of a word.
template <int KIND>
__device__ __forceinline__ uint2 codes_to_half4(uint32_t w) {
  uint2 r;
  if constexpr (KIND == BSA_CACHE_INT8) {
    // 0x64uu is fp16 1024 + u; with u = code + 128: subtract 1152.
    const uint32_t u = w ^ 0x80808080u;
    asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(r.x) : "r"(u), "r"(0x64646464u));
    asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(r.y) : "r"(u), "r"(0x64646464u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"(r.x), "r"(0xe480e480u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r.y) : "r"(r.y), "r"(0xe480e480u));
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
  }
  return r;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Two 2-byte elements (bf16 or fp16) as fp32.
__device__ __forceinline__ float2 elems_to_float2(uint32_t w, bool fp16) {
  if (fp16) return half2_to_float2(w);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

}  // namespace dev
}  // namespace bsa
