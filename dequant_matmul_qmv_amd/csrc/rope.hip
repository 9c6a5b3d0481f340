// Rotary positions: each pair (a, b) of a head turns by the angle
// position * inv_freq[i] into (a cos - b sin, b cos + a sin).  Pairs are
// neighbours (interleaved) or lie rot / 2 apart (halves); dim - rot values
// behind them pass through.
//
// The angle of a far position needs more than 32 bits (131071 rad leaves
// 2^-7 rad of resolution in f32): position * inv_freq / 2 pi is taken in f64,
// its whole turns removed there, and the rest, within half a turn, goes to f32.
//
// Bound: HBM, q and k read once and written once.  One workgroup holds one
// token, computes its rot / 2 cosines and sines once into LDS (every head
// shares them), and walks the heads 16 bytes a lane.
#include "turn_device.h"

namespace mxq {

namespace {

constexpr int kMaxRot = 256;
constexpr double kInvTwoPi = 0.15915494309189533577;

// Cosine and sine of a whole angle, for this token's pairs.
__device__ __forceinline__ void fill_turns(const float* inv_freq, int pos, int half, float* cs, float* sn) {
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double turns = static_cast<double>(pos) * static_cast<double>(inv_freq[i]) * kInvTwoPi;
    const float rest = static_cast<float>(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * rest, &s, &c);
    cs[i] = c;
    sn[i] = s;
  }
  __syncthreads();
}

}  // namespace

// 16-byte rows: dim and rot multiples of 8 (halves: rot of 16).  Units of a
// head: interleaved, dim / 8 chunks; halves, rot / 16 chunks of the first half
// with their partners, then the (dim - rot) / 8 chunks behind.
//
// STREAM: what the call moves does not stay in the L2s anyway, so loads and
// stores pass them by.  8191 tokens of 40 heads of 128 (168 MB, from HBM): 40.4 us
// with loads after the turns, 37.1 with them before, 33.0 (5.1 TB/s, a copy's
// rate) with both.  Called again on one buffer, or on one that was just written,
// part of it comes from the 256 MB cache behind the L2s: 29 .. 32 us.
template <bool BF16, bool INTER, bool STREAM>
__global__ __launch_bounds__(256) void rope_wide_kernel(RopeArgs a) {
  __shared__ float cs[kMaxRot / 2], sn[kMaxRot / 2];
  const int64_t t = blockIdx.x;
  const int half = a.rot / 2;
  const int turned = INTER ? a.rot / 8 : a.rot / 16;
  const int units = turned + (a.dim - a.rot) / 8;
  const int first = a.side[0].heads * units, all = first + a.side[1].heads * units;
  // where unit u lies: its values' offset in the head, and in and out of that head
  struct Unit {
    const uint16_t* in;
    uint16_t* out;
    int c;
    bool turns;
  };
  const auto unit = [&](int u) {
    const RopeSide& s = a.side[u < first ? 0 : 1];
    const int v = u < first ? u : u - first;
    const int head = v / units, c = v - head * units, at = c < turned ? c * 8 : a.rot + (c - turned) * 8;
    return Unit{s.in + t * s.in_token + head * s.in_head + at, s.out + t * s.out_token + head * s.out_head + at, c, c < turned};
  };
  const auto get = [](const uint16_t* p) {
    const u4* v = reinterpret_cast<const u4*>(p);
    if constexpr (STREAM) return __builtin_nontemporal_load(v);
    else return *v;
  };
  const auto put = [](uint16_t* p, u4 x) {
    u4* v = reinterpret_cast<u4*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store(x, v);
    else *v = x;
  };
  const auto load = [&](const Unit& w, u4& lo, u4& hi) {
    lo = get(w.in);
    if constexpr (!INTER)
      if (w.turns) hi = get(w.in + half);
  };
  const auto turn = [&](const Unit& w, u4 lo, u4 hi) {
    if (!w.turns) {
      put(w.out, lo);
    } else if constexpr (INTER) {
      float x[8], y[8];
      widen8<BF16>(lo, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float co = cs[w.c * 4 + i], si = sn[w.c * 4 + i];
        y[2 * i] = x[2 * i] * co - x[2 * i + 1] * si;
        y[2 * i + 1] = x[2 * i + 1] * co + x[2 * i] * si;
      }
      put(w.out, narrow8<BF16>(y));
    } else {
      float x[8], z[8], y[8], v[8];
      widen8<BF16>(lo, x);
      widen8<BF16>(hi, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float co = cs[w.c * 8 + i], si = sn[w.c * 8 + i];
        y[i] = x[i] * co - z[i] * si;
        v[i] = z[i] * co + x[i] * si;
      }
      put(w.out, narrow8<BF16>(y));
      put(w.out + half, narrow8<BF16>(v));
    }
  };
  // the first units are on their way while the turns are computed
  constexpr int kAhead = 3;
  u4 lo[kAhead], hi[kAhead];
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    lo[e] = hi[e] = u4{0, 0, 0, 0};
    const int u = threadIdx.x + e * 256;
    if (u < all) load(unit(u), lo[e], hi[e]);
  }
  fill_turns(a.inv_freq, a.positions[t], half, cs, sn);
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    const int u = threadIdx.x + e * 256;
    if (u < all) turn(unit(u), lo[e], hi[e]);
  }
  for (int u = threadIdx.x + kAhead * 256; u < all; u += 256) {
    const Unit w = unit(u);
    u4 x = u4{0, 0, 0, 0}, z = x;
    load(w, x, z);
    turn(w, x, z);
  }
}

// Any strides, alignments and even rot: one pair, or one value behind them, a lane.
template <bool BF16>
__global__ __launch_bounds__(256) void rope_narrow_kernel(RopeArgs a) {
  __shared__ float cs[kMaxRot / 2], sn[kMaxRot / 2];
  const int64_t t = blockIdx.x;
  const int half = a.rot / 2;
  fill_turns(a.inv_freq, a.positions[t], half, cs, sn);
  const int units = half + a.dim - a.rot;
  const int first = a.side[0].heads * units, all = first + a.side[1].heads * units;
  for (int u = threadIdx.x; u < all; u += blockDim.x) {
    const RopeSide& s = a.side[u < first ? 0 : 1];
    const int v = u < first ? u : u - first;
    const int head = v / units, c = v - head * units;
    const uint16_t* in = s.in + t * s.in_token + head * s.in_head;
    uint16_t* out = s.out + t * s.out_token + head * s.out_head;
    if (c >= half) {
      out[a.rot + c - half] = in[a.rot + c - half];
    } else {
      const int i = a.interleaved ? 2 * c : c, j = a.interleaved ? 2 * c + 1 : half + c;
      const float x = sb_to_f32<BF16>(in[i]), y = sb_to_f32<BF16>(in[j]);
      out[i] = f32_to_act_bits<BF16>(x * cs[c] - y * sn[c]);
      out[j] = f32_to_act_bits<BF16>(y * cs[c] + x * sn[c]);
    }
  }
}

namespace {

constexpr int64_t kL2Bytes = 32 << 20;  // of the eight dies
constexpr int64_t kPartTokens = 1 << 23;  // of a launch, whose grid ends below 2^32 threads

template <bool BF16, bool INTER>
hipError_t launch_wide(const RopeArgs& a) {
  const dim3 grid(static_cast<unsigned>(a.tokens));
  if (4 * a.tokens * (a.side[0].heads + a.side[1].heads) * a.dim > kL2Bytes)
    hipLaunchKernelGGL((rope_wide_kernel<BF16, INTER, true>), grid, dim3(256), 0, a.stream, a);
  else
    hipLaunchKernelGGL((rope_wide_kernel<BF16, INTER, false>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

hipError_t launch_part(const RopeArgs& a) {
  bool wide = a.dim % 8 == 0 && a.rot % (a.interleaved ? 8 : 16) == 0;
  for (const RopeSide& s : a.side)
    if (s.heads > 0)
      wide = wide && ((reinterpret_cast<uintptr_t>(s.in) | reinterpret_cast<uintptr_t>(s.out)) & 15) == 0 &&
             ((s.in_token | s.in_head | s.out_token | s.out_head) & 7) == 0;
  if (wide && a.interleaved) return a.bf16 ? launch_wide<true, true>(a) : launch_wide<false, true>(a);
  if (wide) return a.bf16 ? launch_wide<true, false>(a) : launch_wide<false, false>(a);
  const dim3 grid(static_cast<unsigned>(a.tokens));
  if (a.bf16) hipLaunchKernelGGL((rope_narrow_kernel<true>), grid, dim3(256), 0, a.stream, a);
  else hipLaunchKernelGGL((rope_narrow_kernel<false>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a) {
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kPartTokens) {
    RopeArgs b = a;
    b.tokens = a.tokens - t0 < kPartTokens ? a.tokens - t0 : kPartTokens;
    b.positions += t0;
    for (RopeSide& s : b.side)
      if (s.heads > 0) {
        s.in += t0 * s.in_token;
        s.out += t0 * s.out_token;
      }
    const hipError_t e = launch_part(b);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mxq
