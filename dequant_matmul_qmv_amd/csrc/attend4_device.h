// Device helpers of attention over the 4-bit cache: a value is (c - z) * s, the
// code c and the zero point z of 4 bits, s of 7 significant ones, so every value
// is exact in f16.
#pragma once

#include "attend_split.h"

namespace mxq {

// A word's 8 codes as f16 pairs (c0, c4), (c1, c5), (c2, c6), (c3, c7), each 64 + c: the
// field becomes mantissa bits 4 .. 7 under the exponent of 64.  Seven operations.
// (Codes as the mantissas of subnormal numbers take five, but a product's sums lose
// bits then: 2^-18 of its terms were seen, as if aligned by their exponent fields.)
// Plain code: the compiler knows the wait states that a matrix instruction needs before
// it reads what a vector one wrote; mask and exponent in registers let it use one
// v_and_or_b32.
struct Fields {
  uint32_t mask = 0x00F000F0u, magic = kMagic64;
  __device__ __forceinline__ Fields() { asm("" : "+s"(mask), "+v"(magic)); }
  __device__ __forceinline__ h2 with64(uint32_t bits) const { return as_h2((bits & mask) | magic); }
  __device__ __forceinline__ h8 codes64(uint32_t w) const {
    return as_h8(u4{as_u32(with64(w << 4)), as_u32(with64(w)), as_u32(with64(w >> 4)), as_u32(with64(w >> 8))});
  }
};

// Scales and zero points (as 64 + z) of 8 neighbouring tokens, as pairs in codes' order.
struct Scales8 {
  h2 scale[4], zero64[4];
};
__device__ __forceinline__ Scales8 scales8(const Fields& f, u4 words) {
  const u4 w = perm_x_w4(words);
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
  Scales8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.scale[i] = as_h2(d[i] & 0x7FF07FF0u);
    r.zero64[i] = f.with64(d[i] << 4);
  }
  return r;
}
// c - z of a word of v, and the values of a word, in codes' order: differences of
// codes and products with scales are exact.
__device__ __forceinline__ h8 differences8(const Fields& f, uint32_t w, const Scales8& s) {
  return as_h8(u4{as_u32(f.with64(w << 4) - s.zero64[0]), as_u32(f.with64(w) - s.zero64[1]), as_u32(f.with64(w >> 4) - s.zero64[2]),
                  as_u32(f.with64(w >> 8) - s.zero64[3])});
}
__device__ __forceinline__ h8 values8(const Fields& f, uint32_t w, const Scales8& s) {
  return as_h8(u4{as_u32((f.with64(w << 4) - s.zero64[0]) * s.scale[0]), as_u32((f.with64(w) - s.zero64[1]) * s.scale[1]),
                  as_u32((f.with64(w >> 4) - s.zero64[2]) * s.scale[2]), as_u32((f.with64(w >> 8) - s.zero64[3]) * s.scale[3])});
}

// Scale words of 8 tokens, those from `n` on (n within 16 bits) as zero: where tokens are
// not there, what they hold may be anything.
__device__ __forceinline__ uint32_t pair_below(int i, int n) {
  typedef short s2 __attribute__((ext_vector_type(2)));
  // (the signs of i - n and i + 1 - n, all over their 16 bits: nothing to branch on)
  return __builtin_bit_cast(uint32_t, (s2{static_cast<short>(i), static_cast<short>(i + 1)} - s2{static_cast<short>(n), static_cast<short>(n)}) >> 15);
}
__device__ __forceinline__ u4 first_words(u4 w, int n) {
  return u4{w.x & pair_below(0, n), w.y & pair_below(2, n), w.z & pair_below(4, n), w.w & pair_below(6, n)};
}
// The same for those before `n`.
__device__ __forceinline__ u4 words_from(u4 w, int n) {
  return u4{w.x & ~pair_below(0, n), w.y & ~pair_below(2, n), w.z & ~pair_below(4, n), w.w & ~pair_below(6, n)};
}

}  // namespace mxq
