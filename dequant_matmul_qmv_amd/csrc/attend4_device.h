// Device helpers of attention over the 4-bit cache: a value is (c - z) * s, the
// code c and the zero point z of 4 bits, s of 7 significant ones, so every value
// is exact in f16.
#pragma once

#include "attend_split.h"

namespace mxq {

// A word's 8 codes as f16 pairs (c0, c4), (c1, c5), (c2, c6), (c3, c7), each 2^-24 of
// its value: the field is the mantissa of a subnormal number.
__device__ __forceinline__ h8 codes_tiny(uint32_t w) {
  return as_h8(u4{w & 0x000F000Fu, (w >> 4) & 0x000F000Fu, (w >> 8) & 0x000F000Fu, (w >> 12) & 0x000F000Fu});
}
constexpr float kTinyUnit = 16777216.0f;  // 2^24

// 16 + c of a pair whose codes are in bits 6 .. 9 of each half.
constexpr uint32_t kMagic16 = 0x4C004C00u, kCode16 = 0x03C003C0u;
__device__ __forceinline__ h2 with16(uint32_t bits) { return as_h2(and_or(bits, kCode16, kMagic16)); }

// Scales and zero points of 8 neighbouring tokens, as pairs in codes' order.
struct Scales8 {
  h2 scale[4], zero16[4];  // zero16: 16 + z
};
__device__ __forceinline__ Scales8 scales8(u4 words) {
  const u4 w = perm_x_w4(words);
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
  Scales8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.scale[i] = as_h2(d[i] & 0x7FF07FF0u);
    r.zero16[i] = with16(d[i] << 6);
  }
  return r;
}
// The values of a word, in the same order: differences of codes and products with
// scales are exact.
__device__ __forceinline__ h8 values8(uint32_t w, const Scales8& s) {
  return as_h8(u4{as_u32((with16(w << 6) - s.zero16[0]) * s.scale[0]), as_u32((with16(w << 2) - s.zero16[1]) * s.scale[1]),
                  as_u32((with16(w >> 2) - s.zero16[2]) * s.scale[2]), as_u32((with16(w >> 6) - s.zero16[3]) * s.scale[3])});
}

// Scale words of tokens that are not there (from `n` on, of 8) as zero: what they
// hold may be anything.
__device__ __forceinline__ u4 first_words(u4 w, int n) {
  const auto keep = [n](uint32_t x, int i) { return n >= i + 2 ? x : n > i ? x & 0xFFFFu : 0u; };
  return u4{keep(w.x, 0), keep(w.y, 2), keep(w.z, 4), keep(w.w, 6)};
}

}  // namespace mxq
