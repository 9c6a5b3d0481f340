// Queries and keys normed head by head and rotated by position in one pass:
//
//   y_d = x_d * r * w_d,  r = 1 / sqrt(mean x^2 + eps),
//   (a, b) -> (a cos - b sin, b cos + a sin) for each pair of the first rot values,
//
// a pair's angle being its frequency times the position on its axis (one axis for
// text; time, height and width for frames).
//
// Bound: HBM, q and k read once and written once.  A lane holds 16 values of a
// head, both halves of 8 pairs; dim / 16 neighbours hold the head and add their
// squares by DPP.  A workgroup takes a few tokens: it computes their turns once
// into LDS, where every head reads them, while the first loads are on their way.
#include "turn_device.h"

namespace mxq {

namespace {

constexpr int kMaxDim = 256, kMaxTurns = 512;
constexpr int64_t kL2Bytes = 32 << 20;    // of the eight dies
constexpr int64_t kPartTokens = 1 << 23;  // of a launch, whose grid ends below 2^32 threads

}  // namespace

// 16-byte rows, dim and rot multiples of 16.  STREAM: what the call moves does not
// stay in the L2s anyway, so loads and stores pass them by.
template <bool BF16, bool INTER, bool STREAM>
__global__ __launch_bounds__(256) void norm_rope_wide_kernel(NormRopeArgs a) {
  __shared__ Turn turns[kMaxTurns];
  __shared__ float weights[2][kMaxDim];
  const int half = a.turn.rot / 2, turned = a.turn.rot / 16, used = a.dim / 16;
  const int log2 = used > 8 ? 4 : used > 4 ? 3 : used > 2 ? 2 : used - 1, lanes = 1 << log2;
  const int heads = a.side[0].heads + a.side[1].heads, per = heads << log2, tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.batch;
  const int tokens = a.tokens - t0 < a.batch ? static_cast<int>(a.tokens - t0) : a.batch, all = tokens * per;
  const int c = tid & (lanes - 1);  // the lane's place in its heads
  // its 16-byte pieces there: the two halves of 8 pairs, or neighbours
  const bool turns_here = c < turned;
  const int lo_at = INTER || !turns_here ? 16 * c : 8 * c, hi_at = INTER || !turns_here ? 16 * c + 8 : half + 8 * c;
  struct Unit {
    bool real;
    int tok, side;
    const uint16_t* in;
    uint16_t* out;
  };
  const auto unit = [&](int u) {
    Unit w{u < all && c < used, 0, 0, nullptr, nullptr};
    if (!w.real) return w;
    w.tok = a.batch == 1 ? 0 : u / per;
    int head = (u - w.tok * per) >> log2;
    w.side = head < a.side[0].heads ? 0 : 1;
    const RopeSide& s = a.side[w.side];
    if (w.side == 1) head -= a.side[0].heads;
    w.in = s.in + (t0 + w.tok) * s.in_token + head * s.in_head;
    w.out = s.out + (t0 + w.tok) * s.out_token + head * s.out_head;
    return w;
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
  const bool norms = a.turn.weight[0] != nullptr || a.turn.weight[1] != nullptr;
  const auto turn = [&](const Unit& w, u4 lo, u4 hi) {
    float x[8], z[8];
    widen8<BF16>(lo, x);
    widen8<BF16>(hi, z);
    if (norms) {
      const float r = inverse_norm(group_sum(squares(x) + squares(z), lanes), a.dim, a.turn.eps);
      if (a.turn.weight[w.side] != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = normed(x[i], r, weights[w.side][lo_at + i]);
          z[i] = normed(z[i], r, weights[w.side][hi_at + i]);
        }
      }
    }
    if (!w.real) return;
    if (turns_here) {
      const Turn* t = turns + w.tok * half + 8 * c;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (INTER) {
          float(&y)[8] = i < 4 ? x : z;
          const float p = y[2 * i & 7], q = y[(2 * i & 7) + 1];
          y[2 * i & 7] = turned_first(p, q, t[i]);
          y[(2 * i & 7) + 1] = turned_second(p, q, t[i]);
        } else {
          const float p = x[i], q = z[i];
          x[i] = turned_first(p, q, t[i]);
          z[i] = turned_second(p, q, t[i]);
        }
      }
    }
    put(w.out + lo_at, narrow8<BF16>(x));
    put(w.out + hi_at, narrow8<BF16>(z));
  };
  // the first units are on their way while the turns are computed
  constexpr int kAhead = 2;
  u4 lo[kAhead], hi[kAhead];
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    lo[e] = hi[e] = u4{0, 0, 0, 0};
    const Unit w = unit(tid + e * 256);
    if (w.real) {
      lo[e] = get(w.in + lo_at);
      hi[e] = get(w.in + hi_at);
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (a.turn.weight[s] != nullptr)
      for (int d = tid; d < a.dim; d += 256) weights[s][d] = weight_at<BF16>(a.turn, s, d);
  for (int i = tid; i < tokens * half; i += 256) {
    const int tok = i / half;
    turns[i] = turn_of(a.turn, i - tok * half, t0 + tok, 0);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kAhead; ++e)
    if (e * 256 < all) turn(unit(tid + e * 256), lo[e], hi[e]);
  for (int u0 = kAhead * 256; u0 < all; u0 += 256) {  // whole waves: their lanes add squares
    const Unit w = unit(tid + u0);
    u4 x = u4{0, 0, 0, 0}, z = x;
    if (w.real) {
      x = get(w.in + lo_at);
      z = get(w.in + hi_at);
    }
    turn(w, x, z);
  }
}

// Any strides, alignments, dim and even rot: a wave a head, one token a workgroup.
template <bool BF16>
__global__ __launch_bounds__(256) void norm_rope_narrow_kernel(NormRopeArgs a) {
  __shared__ Turn turns[kMaxDim / 2];
  __shared__ float row[4][kMaxDim];
  const int64_t t = blockIdx.x;
  const int half = a.turn.rot / 2, heads = a.side[0].heads + a.side[1].heads, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < half; i += 256) turns[i] = turn_of(a.turn, i, t, 0);
  for (int h0 = 0; h0 < heads; h0 += 4) {
    const int h = h0 + wave, side = h < a.side[0].heads ? 0 : 1, head = side == 0 ? h : h - a.side[0].heads;
    const bool real = h < heads;
    const RopeSide& s = a.side[side];
    const uint16_t* in = s.in + t * s.in_token + head * s.in_head;
    uint16_t* out = s.out + t * s.out_token + head * s.out_head;
    float x[kMaxDim / 64];
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kMaxDim / 64; ++j) {
      const int d = lane + 64 * j;
      x[j] = real && d < a.dim ? sb_to_f32<BF16>(in[d]) : 0.0f;
      sum = __builtin_fma(static_cast<double>(x[j]), static_cast<double>(x[j]), sum);
    }
    if (a.turn.weight[side] != nullptr) {  // the same for a whole wave
      const float r = inverse_norm(wave_sum(sum), a.dim, a.turn.eps);
#pragma unroll
      for (int j = 0; j < kMaxDim / 64; ++j)
        if (lane + 64 * j < a.dim) x[j] = normed(x[j], r, weight_at<BF16>(a.turn, side, lane + 64 * j));
    }
    __syncthreads();  // the turns; the rows before
#pragma unroll
    for (int j = 0; j < kMaxDim / 64; ++j) row[wave][lane + 64 * j] = x[j];
    __syncthreads();
    if (!real) continue;
#pragma unroll
    for (int j = 0; j < kMaxDim / 64; ++j) {
      const int d = lane + 64 * j;
      if (d >= a.dim) continue;
      float y = x[j];
      if (d < a.turn.rot) {
        const int i = a.turn.interleaved ? d / 2 : d < half ? d : d - half;
        const bool second = a.turn.interleaved ? d & 1 : d >= half;
        const float mate = row[wave][a.turn.interleaved ? d ^ 1 : second ? d - half : d + half];
        y = second ? turned_second(mate, y, turns[i]) : turned_first(y, mate, turns[i]);
      }
      out[d] = f32_to_act_bits<BF16>(y);
    }
  }
}

namespace {

template <bool BF16, bool INTER>
hipError_t launch_wide(const NormRopeArgs& a, unsigned grid) {
  if (4 * a.tokens * (a.side[0].heads + a.side[1].heads) * a.dim > kL2Bytes)
    hipLaunchKernelGGL((norm_rope_wide_kernel<BF16, INTER, true>), dim3(grid), dim3(256), 0, a.stream, a);
  else
    hipLaunchKernelGGL((norm_rope_wide_kernel<BF16, INTER, false>), dim3(grid), dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

hipError_t launch_part(NormRopeArgs a) {
  bool wide = a.dim % 16 == 0 && a.turn.rot % 16 == 0;
  for (const RopeSide& s : a.side)
    if (s.heads > 0)
      wide = wide && ((reinterpret_cast<uintptr_t>(s.in) | reinterpret_cast<uintptr_t>(s.out)) & 15) == 0 &&
             ((s.in_token | s.in_head | s.out_token | s.out_head) & 7) == 0;
  if (!wide) {
    const dim3 grid(static_cast<unsigned>(a.tokens));
    if (a.bf16) hipLaunchKernelGGL((norm_rope_narrow_kernel<true>), grid, dim3(256), 0, a.stream, a);
    else hipLaunchKernelGGL((norm_rope_narrow_kernel<false>), grid, dim3(256), 0, a.stream, a);
    return hipGetLastError();
  }
  a.batch = 1;
  const unsigned grid = static_cast<unsigned>((a.tokens + a.batch - 1) / a.batch);
  if (a.turn.interleaved) return a.bf16 ? launch_wide<true, true>(a, grid) : launch_wide<false, true>(a, grid);
  return a.bf16 ? launch_wide<true, false>(a, grid) : launch_wide<false, false>(a, grid);
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a) {
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kPartTokens) {
    NormRopeArgs b = a;
    b.tokens = a.tokens - t0 < kPartTokens ? a.tokens - t0 : kPartTokens;
    if (b.turn.positions != nullptr) b.turn.positions += t0;
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
