// q8.cuh -- 8-bit floating point (e4m3, e5m2) with power-of-two scales: what
// the fused norm's 8-bit output, the quantisation kernel and the scaled
// matrix product share.
//
// A group is 128 consecutive values of a row (or a 128 x 128 block).  Its
// scale is 2^s with s the smallest integer that brings the group's largest
// magnitude to at most the type's largest finite value, 448 = 1.75 * 2^8
// (e4m3) or 57344 = 1.75 * 2^15 (e5m2); it is held as the byte s + 127, the
// exponent field of 2^s in fp32.  Scaling by a power of two is exact, so the
// one rounding of a value is its conversion to 8 bits (nearest even, half a
// step: 2^-4 relative for e4m3, 2^-3 for e5m2, of a normal result).
#pragma once

#include <stdint.h>

namespace spf {

constexpr int kQ8Group = 128;
constexpr uint32_t kQ8NanScale = 255u;  // the group held Inf or NaN: it stands for NaNs

// Exponent of the largest finite value, 1.75 * 2^kTop.
template <bool E5M2>
struct Q8Top {
  static constexpr int kTop = E5M2 ? 15 : 8;
};

// Scale byte of a group whose largest magnitude has the fp32 bit pattern
// `amax` (sign clear).  With amax = m * 2^(E-127), m in [1, 2): s = E - 127 -
// top, one more when m > 1.75.  Below the smallest scale (fp32 subnormals
// among them) the byte stays 0 and the values round at that scale.
template <bool E5M2>
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return kQ8NanScale;
  if (amax == 0u) return 127u;  // a group of zeros: scale 1
  const int b = (int)(amax >> 23) - Q8Top<E5M2>::kTop + ((amax & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
  return (uint32_t)max(b, 0);
}

// 2^-s for the scale byte s + 127 (bytes 0..247 occur), NaN for the NaN scale.
__device__ __forceinline__ float q8_inv_scale(uint32_t byte) {
  return __uint_as_float(byte == kQ8NanScale ? 0x7FC00000u : (254u - byte) << 23);
}

// 2^s for any scale byte a caller may pass in (byte 0 is the subnormal
// 2^-127, byte 255 is NaN).
__device__ __forceinline__ float q8_scale(uint32_t byte) {
  return __uint_as_float(byte == kQ8NanScale ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Two values to 8 bits, `lo` in the low byte.
template <bool E5M2>
__device__ __forceinline__ uint32_t q8_pack2(float lo, float hi) {
  uint16_t r;
  if constexpr (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  return q8_pack2<E5M2>(a, b) | (q8_pack2<E5M2>(c, d) << 16);
}

// Two 8-bit values (the low 16 bits of w) as fp32, exactly: through fp16,
// which holds every e4m3 and e5m2 value.
__device__ __forceinline__ void q8_unpack2(uint32_t w, bool e5m2, float& lo, float& hi) {
  uint32_t h2;
  const uint16_t v = (uint16_t)w;
  if (e5m2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(v));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(v));
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h2));
}

// max(|a|, |b|, |c|), NaN when one is NaN.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Largest of `v` over the LANES (a power of two) aligned neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

}  // namespace spf
