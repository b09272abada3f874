// The rule by which 4-bit weights (q4.cu) and the 4-bit key/value cache (kv4.cu)
// quantise a group: s = bf16(max |w| / 7), code = clamp(rint(w / s), -7, 7) + 8.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace wc {

// Larger magnitudes (NaN if there is one), with a sign that means nothing.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The BF16 scale of a group whose largest magnitude (BF16 bits, NaN if it
// holds one) is m: the nearest BF16 to m / 7.  m has 8 significant bits, so
// m / 7 is never nearer than 2^-12 of itself to a midpoint of two BF16 values,
// and the rounding of 1 / 7 and of the product cannot cross it.  A group with
// an infinity or a NaN gets the scale NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t m) {
  uint16_t s;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(s) : "f"(__fmul_rn(__uint_as_float(m << 16), 1.f / 7.f)));
  return m >= 0x7F80u ? 0x7FC0u : s;
}

// Code of one weight.  w / s has a quotient of 8-bit significands: it is
// either exactly halfway between integers or at least 2^-10 away from it, so
// w * (1 / s) (2^-22 relative error), rounded to a multiple of 2^-12 by the
// first constant, is on the right side of every halfway point, and exactly on
// it where w / s is; the second, added less the first (both sums are exact but for
// the one rounding to a whole number), then rounds half to even.  Scales
// below 2^-100 (reciprocals near overflow, quotients above 7) divide and clamp.
constexpr float kSnap = 0x1.8p11f;        // 1.5 * 2^11: ulp 2^-12
// Codes come as kBase + code, so that a word of eight is a sum of them times
// powers of 16, less what the bases add up to: one integer multiply-add a code.
constexpr float kRound = 12582920.f;   // 1.5 * 2^23 + 8: ulp 1, and the code's offset of 8
constexpr uint32_t kBase = 0x4B400000u;  // the bits of 1.5 * 2^23
__device__ __forceinline__ uint32_t code_fast(float w, float rs) {
  return __float_as_uint(__fadd_rn(__fmaf_rn(w, rs, kSnap), kRound - kSnap));
}
__device__ __forceinline__ uint32_t code_slow(float w, float s) {
  if (!(s > 0.f)) return 8u;  // scale 0 or NaN
  return uint32_t(int(fminf(fmaxf(rintf(__fdiv_rn(w, s)), -7.f), 7.f)) + 8);
}

__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

}  // namespace wc
