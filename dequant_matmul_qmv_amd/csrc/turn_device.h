// Norms and rotary turns of heads, shared by the kernels that have to agree on
// their bits: cosines, sines and inverse norms are taken in f64 and rounded once
// to f32, every product and sum after them is an f32 operation of its own (no
// fused multiply-add), and the result is rounded once to the storage type.
#pragma once

#include "lanes_device.h"
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

template <bool BF16>
__device__ __forceinline__ void widen8(u4 v, float (&f)[8]) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = sb_to_f32<BF16>(static_cast<uint16_t>(d[i]));
    f[2 * i + 1] = sb_to_f32<BF16>(static_cast<uint16_t>(d[i] >> 16));
  }
}

template <bool BF16>
__device__ __forceinline__ u4 narrow8(const float (&f)[8]) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d[i] = static_cast<uint32_t>(f32_to_act_bits<BF16>(f[2 * i])) |
           (static_cast<uint32_t>(f32_to_act_bits<BF16>(f[2 * i + 1])) << 16);
  return u4{d[0], d[1], d[2], d[3]};
}

// Cosine and sine of a pair's angle.
struct __align__(8) Turn {
  float c, s;
};

// The angle, position * frequency, less a multiple of pi / 2 (held in two parts:
// 106 bits), then the Taylor series of sine and cosine on [-pi/4, pi/4], whose
// first terms left out are below 2^-53.  About 40 f64 operations, which run at
// the rate of f32 here.
__device__ __forceinline__ Turn turn_by(int pos, float inv_freq) {
  constexpr double kQuarters = 0.63661977236758134308;  // 2 / pi
  constexpr double kQuarter = 1.5707963267948965580, kQuarterRest = 6.1232339957367660359e-17;
  const double angle = static_cast<double>(pos) * static_cast<double>(inv_freq);
  const double k = __builtin_rint(angle * kQuarters);
  const double r = __builtin_fma(-k, kQuarterRest, __builtin_fma(-k, kQuarter, angle)), q = r * r;
  double s = -1.0 / 1307674368000.0;
  s = __builtin_fma(s, q, 1.0 / 6227020800.0);
  s = __builtin_fma(s, q, -1.0 / 39916800.0);
  s = __builtin_fma(s, q, 1.0 / 362880.0);
  s = __builtin_fma(s, q, -1.0 / 5040.0);
  s = __builtin_fma(s, q, 1.0 / 120.0);
  s = __builtin_fma(s, q, -1.0 / 6.0);
  s = __builtin_fma(s * q, r, r);
  double c = 1.0 / 20922789888000.0;
  c = __builtin_fma(c, q, -1.0 / 87178291200.0);
  c = __builtin_fma(c, q, 1.0 / 479001600.0);
  c = __builtin_fma(c, q, -1.0 / 3628800.0);
  c = __builtin_fma(c, q, 1.0 / 40320.0);
  c = __builtin_fma(c, q, -1.0 / 720.0);
  c = __builtin_fma(c, q, 1.0 / 24.0);
  c = __builtin_fma(c, q, -0.5);
  c = __builtin_fma(c, q, 1.0);
  const int quadrant = static_cast<int>(k - 4.0 * __builtin_rint(k * 0.25)) & 3;
  const float fs = static_cast<float>(s), fc = static_cast<float>(c);
  const float co = quadrant & 1 ? fs : fc, si = quadrant & 1 ? fc : fs;
  return Turn{quadrant == 1 || quadrant == 2 ? -co : co, quadrant >= 2 ? -si : si};
}

// What pair i's turn of row t is made of; `place` is the row's place in its sequence.
// Loads are answered in order, so these come before those of the rows: the turn is then
// computed while the rows are on their way.
struct TurnInput {
  int pos;
  float inv_freq;
  __device__ __forceinline__ Turn turn() const { return turn_by(pos, inv_freq); }
};
__device__ __forceinline__ TurnInput turn_input(const TurnArgs& a, int i, int64_t t, int place) {
  const int axis = a.axis != nullptr ? min(max(a.axis[i], 0), a.axes - 1) : 0;
  return TurnInput{a.positions != nullptr ? a.positions[axis * a.axis_stride + t] : place, a.inv_freq[i]};
}
__device__ __forceinline__ Turn turn_of(const TurnArgs& a, int i, int64_t t, int place) { return turn_input(a, i, t, place).turn(); }

// Eight f32 values rounded to storage.  (The values are made opaque: a sum and its
// rounding must not become one operation.)
template <bool BF16>
__device__ __forceinline__ u4 round8(const float (&f)[8]) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = f[2 * i], y = f[2 * i + 1];
    asm("" : "+v"(x), "+v"(y));
    if constexpr (BF16) {
      d[i] = pack_bf16_pair(x, y);
    } else {
      const h2 p = {static_cast<_Float16>(x), static_cast<_Float16>(y)};
      d[i] = as_u32(p);
    }
  }
  return u4{d[0], d[1], d[2], d[3]};
}

// f32(1 / sqrt(sum / dim + eps)): the instruction's estimate and two steps of
// Newton's iteration in f64.
__device__ __forceinline__ float inverse_norm(double sum, double inv_dim, double eps) {
  const double m = __builtin_fma(sum, inv_dim, eps);
  double y = __builtin_amdgcn_rsq(m);
  if (m > 0.0 && m < __builtin_inf()) {
#pragma unroll
    for (int i = 0; i < 2; ++i) y = __builtin_fma(0.5 * y, __builtin_fma(-m * y, y, 1.0), y);
  }
  return static_cast<float>(y);
}

// Sum over groups of `lanes` neighbours (1, 2, 4, 8 or 16), the same in each of them.
__device__ __forceinline__ double group_sum(double x, int lanes) {
  if (lanes > 1) x += lane_move<0xB1, 0xF>(x);   // lane ^ 1, lane ^ 2
  if (lanes > 2) x += lane_move<0x4E, 0xF>(x);
  if (lanes > 4) x += lane_move<0x141, 0xF>(x);  // 7 - lane, 15 - lane of 8 and 16
  if (lanes > 8) x += lane_move<0x140, 0xF>(x);
  return x;
}
__device__ __forceinline__ double squares(const float (&x)[8]) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fma(static_cast<double>(x[i]), static_cast<double>(x[i]), s);
  return s;
}

// x * r * w, and the first and second value of a turned pair.
__device__ __forceinline__ float normed(float x, float r, float w) {
#pragma clang fp contract(off)
  const float y = x * r;
  return y * w;
}
__device__ __forceinline__ float turned_first(float a, float b, Turn t) {
#pragma clang fp contract(off)
  const float x = a * t.c, y = b * t.s;
  return x - y;
}
__device__ __forceinline__ float turned_second(float a, float b, Turn t) {
#pragma clang fp contract(off)
  const float x = b * t.c, y = a * t.s;
  return x + y;
}

// A lane's 16-byte pieces of a head of 16 * `used` values, of which it is lane c: the two
// halves of 8 pairs; interleaved, two that neighbours' pieces lie beside; behind the turned
// part, neighbours.  rot is a multiple of 16.
struct HeadLane {
  int lo, hi;
  bool lo_turns, hi_turns;  // hi_turns: interleaved; the halves turn together
};
template <bool INTER>
__device__ __forceinline__ HeadLane head_lane(int c, int used, int rot) {
  const bool turned = c < rot / 16;
  HeadLane l;
  l.lo = INTER || turned ? 8 * c : 16 * c;
  l.hi = INTER ? 8 * (used + c) : turned ? rot / 2 + 8 * c : 16 * c + 8;
  l.lo_turns = INTER ? l.lo < rot : turned;
  l.hi_turns = INTER && l.hi < rot;
  return l;
}
// Its values turned, by the row's table.
template <bool INTER>
__device__ __forceinline__ void turn16(float (&x)[8], float (&z)[8], const HeadLane& l, const Turn* t) {
  if constexpr (INTER) {
    const auto turn4 = [](float(&y)[8], const Turn* by) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float p = y[i], q = y[i + 1];
        y[i] = turned_first(p, q, by[i / 2]);
        y[i + 1] = turned_second(p, q, by[i / 2]);
      }
    };
    if (l.lo_turns) turn4(x, t + l.lo / 2);
    if (l.hi_turns) turn4(z, t + l.hi / 2);
  } else if (l.lo_turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = x[i], q = z[i];
      x[i] = turned_first(p, q, t[l.lo + i]);
      z[i] = turned_second(p, q, t[l.lo + i]);
    }
  }
}

// A side's weights.  (A side that differs by lane must not index the arguments: they would
// be copied to scratch memory, and every pointer in them with them.)
__device__ __forceinline__ const void* side_weight(const TurnArgs& a, int side) { return side == 0 ? a.weight[0] : a.weight[1]; }
// Norm weight d in f32.
template <bool BF16>
__device__ __forceinline__ float weight_at(const TurnArgs& a, int side, int d) {
  if (a.weight_f32) return static_cast<const float*>(side_weight(a, side))[d];
  return sb_to_f32<BF16>(static_cast<const uint16_t*>(side_weight(a, side))[d]);
}
// Eight of them, from a multiple of 8 on.
template <bool BF16>
__device__ __forceinline__ void weights8(const TurnArgs& a, int side, int d, float (&w)[8]) {
  if (!a.weight_wide) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = weight_at<BF16>(a, side, d + i);
  } else if (a.weight_f32) {
    typedef float f4 __attribute__((ext_vector_type(4)));
    const f4* p = reinterpret_cast<const f4*>(static_cast<const float*>(side_weight(a, side)) + d);
    const f4 x = p[0], y = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i], w[4 + i] = y[i];
  } else {
    widen8<BF16>(*reinterpret_cast<const u4*>(static_cast<const uint16_t*>(side_weight(a, side)) + d), w);
  }
}

}  // namespace mxq
