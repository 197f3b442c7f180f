// e4m3.cuh -- the number format of the 8-bit cache, shared by its write, its
// read-back and the decode over it.
//
// A row x of d_h numbers (one token of one KV head) is held as d_h e4m3 codes
// and one biased exponent byte E: value = code * 2^(E - 127). With a the
// largest finite |x|, e = E - 127 is the smallest exponent in [-117, 119] with
// a <= 448 * 2^e (448: the largest e4m3 number), and code = e4m3(x * 2^-e),
// ties to even. The scale is a power of two, so x * 2^-e and code * 2^e are
// exact: the one rounding is that to e4m3, the code of a value does not depend
// on how the scale is applied, and every stored value is a bf16 number. (A
// scale of a / 448 would use up to one more bit of e4m3's range, but e4m3 is a
// floating format: its relative step is the same at 224 as at 448.) The limits
// keep 2^e, 2^-e and every stored value normal in bf16 and fp32.
#pragma once

#include <stdint.h>

namespace attn {
namespace e4m3 {

constexpr int kPage = 16;
constexpr int kExpMin = -117, kExpMax = 119;

// Biased exponent byte for a row whose largest finite magnitude has the fp32
// bits `abits`. 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_byte(uint32_t abits) {
  int e = static_cast<int>(abits >> 23) - 127 - 8 + ((abits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(kExpMin, min(kExpMax, e));
  return static_cast<uint32_t>(e + 127);
}

// 2^(byte - 127) (bytes of a well-formed cache lie in [10, 246]) and, for
// those, its inverse.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float inv_scale_of(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Two e4m3 codes (low byte first) of a pair of fp32 numbers; beyond 448 the
// largest code, NaN stays NaN.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes (low byte first) as a pair of fp16 numbers: exact, every e4m3
// number is an fp16 number.
__device__ __forceinline__ uint32_t decode2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

}  // namespace e4m3
}  // namespace attn
