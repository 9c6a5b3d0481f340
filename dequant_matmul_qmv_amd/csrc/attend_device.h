// Device helpers shared by the attention kernels over the 8-bit cache.
#pragma once

#include "lanes_device.h"
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

typedef float f4 __attribute__((ext_vector_type(4)));

// Eight int8 codes as exact f16: each byte, offset to c + 128, becomes the
// mantissa of 1024 (0x6400 | u), and -1152 leaves c: 5 operations for 4 codes.
__device__ __forceinline__ u4 codes8_f16(uint32_t w0, uint32_t w1, uint32_t magic) {
  const h2 off = {static_cast<_Float16>(-1152.0f), static_cast<_Float16>(-1152.0f)};
  w0 ^= 0x80808080u;
  w1 ^= 0x80808080u;
  const uint32_t lo = 0x05010500u, hi = 0x05030502u;
  return u4{as_u32(as_h2(__builtin_amdgcn_perm(magic, w0, lo)) + off), as_u32(as_h2(__builtin_amdgcn_perm(magic, w0, hi)) + off),
            as_u32(as_h2(__builtin_amdgcn_perm(magic, w1, lo)) + off), as_u32(as_h2(__builtin_amdgcn_perm(magic, w1, hi)) + off)};
}

__device__ __forceinline__ h8 as_h8(u4 v) { return __builtin_bit_cast(h8, v); }

// x of lane ^ 32, lane ^ 16 combined with the own, by VALU row swaps.
__device__ __forceinline__ float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

constexpr float kNegInf = -__builtin_inff();
// Probabilities are held as 2^kLift times their value: f16 then keeps full
// precision down to 2^-28 of a row's largest one.
constexpr float kLift = 14.0f;
constexpr float kF16Normal = 6.103515625e-05f;  // 2^-14, f16's smallest normal value
constexpr float kLowLift = 16777216.0f;         // 2^24
constexpr float kUnlift = 1.0f / 16384.0f;

// Weights below f16's normal range go through products of their own, a band of
// 2^24 at a time, each lifted into that range.  The fifth band ends at 2^-134
// (an f32 weight times its page's share of the largest v scale can be smaller):
// what is below, 2^-148 of the row's largest weight times the largest v scale,
// is dropped, since a sixth lift would be past f32's range.
struct Band {
  float ceiling = kF16Normal, floor = kF16Normal / kLowLift, lift = kLowLift;
  __device__ __forceinline__ float lifted(float p) const { return p < ceiling && p >= floor ? p * lift : 0.0f; }
  __device__ __forceinline__ bool below(float p) const { return p > 0.0f && p < floor; }
  __device__ __forceinline__ bool last() const { return lift >= 0x1p120f; }
  __device__ __forceinline__ void next() {
    ceiling = floor;
    floor *= 1.0f / kLowLift;
    lift *= kLowLift;
  }
};
constexpr float kLn2 = 0.69314718055994530942f;
// One over a row's weight; 0 for a row without keys.
__device__ __forceinline__ float over(float total) { return total > 0.0f || total != total ? 1.0f / total : 0.0f; }
// A row's parts are kept divided by their weight, and joined by their weights
// times this: sums of values near f32's largest or smallest stay in its range.
constexpr float kJoinUnit = 1.0f / kLowLift;
// Natural log-sum of weights held as 2^kLift times 2^(x - ref).
__device__ __forceinline__ float log_sum(float ref, float total) { return (ref + log2f(total * kUnlift)) * kLn2; }

// Eight values of a query row in f16.  f16 rows as stored; bf16 rows are taken
// times 2^-e, e the exponent of the row's largest magnitude: f16 then holds
// every value to 2^-25 of the largest, and e goes into the softmax's scale.
__device__ __forceinline__ u4 bf16_to_scaled_f16(u4 v, float factor) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const h2 r = {static_cast<_Float16>(__uint_as_float(d[i] << 16) * factor),
                  static_cast<_Float16>(__uint_as_float(d[i] & 0xFFFF0000u) * factor)};
    o[i] = as_u32(r);
  }
  return u4{o[0], o[1], o[2], o[3]};
}

// A power of two that brings `top` (a bf16 row's largest magnitude) near 1 (to
// [1, 4); below it for rows under bf16's normal range), and its inverse.  Zero,
// infinite and NaN rows keep 1.
__device__ __forceinline__ void row_factor(float top, float& factor, float& inverse) {
  // 2^(127-e) stays a normal number for e of 1 .. 253
  const uint32_t e = min(max((__float_as_uint(top) >> 23) & 0xFFu, 1u), 253u);
  const bool fine = top > 0.0f && top < __builtin_inff();
  factor = fine ? __uint_as_float((254u - e) << 23) : 1.0f;
  inverse = fine ? __uint_as_float(e << 23) : 1.0f;
}

__device__ __forceinline__ float absmax8_bf16(u4 v) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(d[i] << 16)), fabsf(__uint_as_float(d[i] & 0xFFFF0000u))));
  return m;
}

// A sequence's part of the call: its new rows of q, and its length.
struct SeqSpan {
  int t0, n, len;
};
__device__ __forceinline__ SeqSpan seq_span(const AttendArgs& a, int s) {
  SeqSpan r;
  if (a.starts == nullptr) {
    r.t0 = s;
    r.n = 1;
  } else {
    r.t0 = min(max(a.starts[s], 0), a.tokens);
    r.n = min(max(a.starts[s + 1], r.t0), a.tokens) - r.t0;
  }
  r.len = max(a.lens[s], 0);
  return r;
}

// The first key that a token at `pos` sees (negative positions see none; a
// window up to 2^31 - 1 must not wrap there).
__device__ __forceinline__ int first_seen(const AttendArgs& a, int pos) { return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0; }

}  // namespace mxq
