// Queries and keys normed head by head and rotated by position in one pass:
//
//   y_d = x_d * r * w_d,  r = 1 / sqrt(mean x^2 + eps),
//   (a, b) -> (a cos - b sin, b cos + a sin) for each pair of the first rot values,
//
// a pair's angle being its frequency times the position on its axis (one axis for
// text; time, height and width for frames).
//
// Bound: HBM, q and k read once and written once, with the vector ALU close behind (a
// mean of squares in f64, two products and a turn for each value).  A lane holds 16
// values of a head, both halves of 8 pairs; dim / 16 neighbours hold the head and add
// their squares by DPP.  A lane keeps its place in the token, and its weights, for all
// of the workgroup's tokens, and loads the next token's values before it turns one; the
// turns of all of them are computed once into LDS, while the first loads are on their way.
#include "turn_device.h"

namespace mxq {

namespace {

constexpr int kMaxDim = 256, kMaxTurns = 1024;
constexpr int kMostThreads = 512;
// Workgroups of a long call, two for each compute unit: what a workgroup does before its
// first token costs as much as 1.5 tokens of 40 heads (8191 of them: 75 us with one token a
// workgroup, 53 with two, 36.5 with 4, 39.2 with 8, 35.5 with 16, those of two whole rounds).
constexpr int kWorkgroups = 512;
constexpr int64_t kL2Bytes = 32 << 20;    // of the eight dies
constexpr int64_t kPartTokens = 1 << 23;  // of a launch, whose grid ends below 2^32 threads

}  // namespace

// 16-byte rows, dim and rot multiples of 16.  STREAM: what the call moves does not
// stay in the L2s anyway, so loads and stores pass them by.
template <bool BF16, bool INTER, bool STREAM>
__global__ __launch_bounds__(kMostThreads) void norm_rope_wide_kernel(NormRopeArgs a) {
  __shared__ Turn turns[kMaxTurns];
  const int half = a.turn.rot / 2, used = a.dim / 16;
  const int log2 = used > 8 ? 4 : used > 4 ? 3 : used > 2 ? 2 : used - 1, lanes = 1 << log2;
  const int heads = a.side[0].heads + a.side[1].heads, per = heads << log2, tid = threadIdx.x;
  // the lane's place: its token of those that the workgroup has at a time, its head and
  // its pieces there
  const int place = static_cast<int>(blockIdx.y) * kMostThreads + tid;
  // (one lane a token: 1 has no inverse below 2^32)
  const int sub = a.abreast == 1 ? 0 : per == 1 ? place : static_cast<int>(__umulhi(place, a.per_inverse));
  const int slot = place - sub * per, c = slot & (lanes - 1);
  int head = slot >> log2;
  const bool here = head < heads && sub < a.abreast && c < used;
  const int side = head < a.side[0].heads ? 0 : 1;
  if (side == 1) head -= a.side[0].heads;
  const HeadLane at = head_lane<INTER>(c, used, a.turn.rot);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.batch;
  const int tokens = a.tokens - t0 < a.batch ? static_cast<int>(a.tokens - t0) : a.batch;
  const RopeSide s = side == 0 ? a.side[0] : a.side[1];
  const uint16_t* in = s.in + (t0 + sub) * s.in_token + head * s.in_head;
  uint16_t* out = s.out + (t0 + sub) * s.out_token + head * s.out_head;
  const int64_t in_step = a.abreast * s.in_token, out_step = a.abreast * s.out_token;
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
  // loads are answered in order: those of the first turn and of the weights come first
  TurnInput mine{0, 0.0f};
  const int all_turns = tokens * half;
  const auto input = [&](int i) {
    const int tok = static_cast<int>(__umulhi(i, a.half_inverse));
    return turn_input(a.turn, i - tok * half, t0 + tok, 0);
  };
  if (tid < all_turns) mine = input(tid);
  const bool norm = side_weight(a.turn, side) != nullptr && here, norms = a.turn.weight[0] != nullptr || a.turn.weight[1] != nullptr;
  float wx[8], wz[8];
  if (norm) {
    weights8<BF16>(a.turn, side, at.lo, wx);
    weights8<BF16>(a.turn, side, at.hi, wz);
  }
  u4 lo = u4{0, 0, 0, 0}, hi = lo;
  if (here && sub < tokens) {
    lo = get(in + at.lo);
    hi = get(in + at.hi);
  }
  if (tid < all_turns) turns[tid] = mine.turn();
  for (int i = tid + blockDim.x; i < all_turns; i += blockDim.x) turns[i] = input(i).turn();
  __syncthreads();
  const Turn* t = turns + sub * half;
  for (int tok = sub; tok - sub < tokens; tok += a.abreast) {  // whole waves: their lanes add squares
    float x[8], z[8];
    widen8<BF16>(lo, x);
    widen8<BF16>(hi, z);
    in += in_step;
    if (here && tok + a.abreast < tokens) {
      lo = get(in + at.lo);
      hi = get(in + at.hi);
    }
    if (norms) {
      const float r = inverse_norm(group_sum(squares(x) + squares(z), lanes), a.turn.inv_dim, a.turn.eps);
      if (norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = normed(x[i], r, wx[i]);
          z[i] = normed(z[i], r, wz[i]);
        }
      }
    }
    if (here && tok < tokens) {
      turn16<INTER>(x, z, at, t);
      put(out + at.lo, round8<BF16>(x));
      put(out + at.hi, round8<BF16>(z));
    }
    out += out_step;
    t += a.abreast * half;
  }
}

// Any strides, alignments, dim and even rot: a wave a head, one token a workgroup, 2 bytes
// an access (8191 tokens of 40 heads of 128: 117 us, the wide kernel 35).
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
    const RopeSide s = side == 0 ? a.side[0] : a.side[1];
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
    if (side_weight(a.turn, side) != nullptr) {  // the same for a whole wave
      const float r = inverse_norm(wave_sum(sum), a.turn.inv_dim, a.turn.eps);
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
hipError_t launch_wide(const NormRopeArgs& a, dim3 grid, dim3 block) {
  if (4 * a.tokens * (a.side[0].heads + a.side[1].heads) * a.dim > kL2Bytes)
    hipLaunchKernelGGL((norm_rope_wide_kernel<BF16, INTER, true>), grid, block, 0, a.stream, a);
  else
    hipLaunchKernelGGL((norm_rope_wide_kernel<BF16, INTER, false>), grid, block, 0, a.stream, a);
  return hipGetLastError();
}

// ceil(2^32 / d): __umulhi with it divides numbers up to 2^16 by d of 2 up to 2^12 (of 1 it
// would be 2^32: the kernel does not divide there).
uint32_t over32(int d) { return static_cast<uint32_t>(((uint64_t{1} << 32) + d - 1) / d); }

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
  // tokens abreast: as many as fill whole waves best; then as many times those as leave
  // each compute unit several workgroups
  const int half = a.turn.rot / 2, used = a.dim / 16, lanes = used > 8 ? 16 : used > 4 ? 8 : used > 2 ? 4 : used;
  const int per = (a.side[0].heads + a.side[1].heads) * lanes;
  a.abreast = 1;
  int threads = (per + 63) / 64 * 64;
  for (int n = 2; n * per <= kMostThreads && n * int64_t{512} <= a.tokens; ++n) {
    const int t = (n * per + 63) / 64 * 64;
    if (static_cast<int64_t>(n) * threads > static_cast<int64_t>(a.abreast) * t) {
      a.abreast = n;
      threads = t;
    }
  }
  int64_t times = (a.tokens + a.abreast * int64_t{kWorkgroups} - 1) / (a.abreast * int64_t{kWorkgroups});
  if (times > 16) times = 16;
  if (times * a.abreast * half > kMaxTurns) times = kMaxTurns / (a.abreast * half);
  a.batch = a.abreast * static_cast<int>(times < 1 ? 1 : times);
  a.per_inverse = over32(per);
  a.half_inverse = half > 0 ? over32(half) : 0;
  const dim3 grid(static_cast<unsigned>((a.tokens + a.batch - 1) / a.batch), static_cast<unsigned>((threads + kMostThreads - 1) / kMostThreads));
  const dim3 block(static_cast<unsigned>(threads < kMostThreads ? threads : kMostThreads));
  if (a.turn.interleaved) return a.bf16 ? launch_wide<true, true>(a, grid, block) : launch_wide<false, true>(a, grid, block);
  return a.bf16 ? launch_wide<true, false>(a, grid, block) : launch_wide<false, false>(a, grid, block);
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
