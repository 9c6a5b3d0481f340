// New keys normed, rotated and quantized into a paged cache of 8 or 4 bits with
// the new values, and queries normed and rotated beside them: the way from the
// fused projection's output to attention in one launch.
//
// Keys are rounded to their type after the turn, so the codes are those of a norm
// and rotation into memory with an append after it.  The scheme of 8 bits is that
// of the plain append.  4 bits hold (c - z) * s: s a fifteenth of a token and
// head's range, zero within it, up to the next number of 7 significant bits; 4
// bits times 7 are exact in f16, so attention's products have exact operands.  A
// scale and its zero point share a 16-bit word, f16 with z as its lowest bits.
// A quotient is taken in f64 and rounded to f32 once.
//
// Bound: the vector ALU and HBM for prompts (4 bits, 224 MB in 53 us: 4.2 TB/s; without
// norms 181 MB in 38), dependent loads for single tokens (lens, table, scale or words: 64
// tokens into 4 bits 6.0 us) and, for 8 bits, v's stores of a byte to a line (256 tokens 10.6).
#include "append_device.h"
#include "turn_device.h"

namespace mxq {

namespace {

constexpr int kMaxHead = 128, kGroup = 8;  // values of a head; tokens that share a word of v
constexpr float kMaxScale4 = 4064.0f;      // 16 times it is within f16's range
constexpr int kOneThreads = 256;           // at most, of a single token's kv head
constexpr int kGroupThreads = 512;         // a wave for each of a group's 8 places

// A piece of 8 values of a head, and the values they turn with.
struct Piece {
  u4 own, mate;
};

// What the turns of a workgroup's rows are made of: LDS tables of theirs and of
// the norms' weights.
//
// MODE kAnyRows: any alignment, rot and order of pairs (5 prompts into 4 bits 117 us, into 8
// bits 25, aligned 58 and 12); else rows that are 16-byte
// aligned with rot a multiple of 16, whose pieces turn as a whole or not at all: halves,
// or interleaved pairs.
enum { kAnyRows, kHalves, kPairs };
template <int MODE>
struct Turner {
  const TurnArgs* turn;
  const Turn* turns;               // [rows][rot / 2]
  const float (*weights)[kMaxHead];  // of q, of k
  int dim, half;

  // Where the value that d turns with lies (itself beyond the turned part).
  __device__ __forceinline__ int mate_of(int d) const { return d < half ? d + half : d < 2 * half ? d - half : d; }
  __device__ __forceinline__ Piece load(const uint16_t* x, int c, bool wide) const {
    Piece p;
    if constexpr (MODE != kAnyRows) {
      p.own = p.mate = load16(x + c * 8, true);
      if (MODE == kHalves && c * 8 < 2 * half) p.mate = load16(x + mate_of(c * 8), true);
    } else {
      p.own = p.mate = load16(x + c * 8, wide);
      if (!turn->interleaved && c * 8 < 2 * half) {
        uint32_t d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d[j] = static_cast<uint32_t>(x[mate_of(c * 8 + 2 * j)]) | (static_cast<uint32_t>(x[mate_of(c * 8 + 2 * j + 1)]) << 16);
        p.mate = u4{d[0], d[1], d[2], d[3]};
      }
    }
    return p;
  }
  // Whole waves: the dim / 8 lanes of a head add their squares.
  template <bool BF16>
  __device__ __forceinline__ u4 finish(const Piece& p, int row, int c, int side) const {
    float x[8], z[8];
    widen8<BF16>(p.own, x);
    widen8<BF16>(p.mate, z);
    if (turn->weight[0] != nullptr || turn->weight[1] != nullptr) {  // (the same in the whole wave)
      const float r = inverse_norm(group_sum(squares(x), dim / 8), turn->inv_dim, turn->eps);
      if (side_weight(*turn, side) != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = normed(x[j], r, weights[side][c * 8 + j]);
          if (MODE != kPairs) z[j] = normed(z[j], r, weights[side][mate_of(c * 8 + j)]);
        }
      }
    }
    float y[8];
    const int first = c * 8;
    if constexpr (MODE != kAnyRows) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[j];
      if (first < 2 * half) {
        if constexpr (MODE == kPairs) {
          const Turn* t = turns + row * half + first / 2;
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            y[j] = turned_first(x[j], x[j + 1], t[j / 2]);
            y[j + 1] = turned_second(x[j], x[j + 1], t[j / 2]);
          }
        } else {
          // (a sum with the negative is the difference, bit for bit)
          const Turn* t = turns + row * half + (first < half ? first : first - half);
          const uint32_t sign = first < half ? 0x80000000u : 0u;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            y[j] = turned_second(z[j], x[j], Turn{t[j].c, __uint_as_float(__float_as_uint(t[j].s) ^ sign)});
        }
      }
      return round8<BF16>(y);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = first + j;
      y[j] = x[j];
      if (d >= 2 * half) continue;
      if (turn->interleaved) {
        const Turn t = turns[row * half + d / 2];
        y[j] = j & 1 ? turned_second(x[j ^ 1], x[j], t) : turned_first(x[j], x[j ^ 1], t);
      } else {
        const Turn t = turns[row * half + (d < half ? d : d - half)];
        y[j] = d < half ? turned_first(x[j], z[j], t) : turned_second(z[j], x[j], t);
      }
    }
    return round8<BF16>(y);
  }
};

__device__ __forceinline__ void store16(uint16_t* p, u4 v, bool wide) {
  if (wide) {
    *reinterpret_cast<u4*>(p) = v;
    return;
  }
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[2 * i] = static_cast<uint16_t>(d[i]);
    p[2 * i + 1] = static_cast<uint16_t>(d[i] >> 16);
  }
}

template <bool BF16>
__device__ __forceinline__ void fill_weights(const TurnArgs& t, int dim, float (*weights)[kMaxHead]) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (t.weight[s] != nullptr)
      for (int d = threadIdx.x; d < dim; d += blockDim.x) weights[s][d] = weight_at<BF16>(t, s, d);
}

// Largest of a head's `lanes` lanes (4, 8 or 16).
__device__ __forceinline__ float group_max(float x, int lanes) {
  x = fmaxf(x, lane_move<0xB1, 0xF>(x));
  x = fmaxf(x, lane_move<0x4E, 0xF>(x));
  if (lanes > 4) x = fmaxf(x, lane_move<0x141, 0xF>(x));
  if (lanes > 8) x = fmaxf(x, lane_move<0x140, 0xF>(x));
  return x;
}

// ---- 4 bits
// The scale and zero point of values within lo <= 0 <= hi.
struct Scaling4 {
  float inv, zero;
  uint16_t word;
};
__device__ __forceinline__ Scaling4 scaling4(float lo, float hi) {
  // range / 15 correctly rounded: a product with the rounded inverse, mended by the exact
  // rest (Markstein)
  const double range = static_cast<double>(hi) - static_cast<double>(lo), fifteenth = 1.0 / 15.0;
  const double near = range * fifteenth, step = __builtin_fma(__builtin_fma(-15.0, near, range), fifteenth, near);
  const int unit = max(__builtin_amdgcn_frexp_exp(step) - 7, -20);  // 7 bits, and f16's subnormal ones less 4
  const double up = __builtin_ldexp(__builtin_ceil(__builtin_ldexp(step, -unit)), unit);
  const float scale = fminf(static_cast<float>(up), kMaxScale4);
  Scaling4 s{0.0f, 0.0f, 0};
  // 1 / scale correctly rounded in the same way: a scale has one of 64 mantissas, and all
  // of them are tested
  const float inv = __builtin_amdgcn_rcpf(scale);
  if (scale > 0.0f) s.inv = __builtin_fmaf(__builtin_fmaf(-scale, inv, 1.0f), inv, inv);
  s.zero = fminf(__builtin_rintf(-lo * s.inv), 15.0f);
  s.word = static_cast<uint16_t>(f32_to_f16_bits(scale) | static_cast<uint16_t>(s.zero));
  return s;
}
template <bool BF16>
__device__ __forceinline__ Scaling4 scaling4_of(u4 v, int lanes) {
  float x[8];
  widen8<BF16>(v, x);
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
  return scaling4(-group_max(-lo, lanes), group_max(hi, lanes));
}
__device__ __forceinline__ void codes4(const float (&x)[8], const Scaling4& s, uint32_t (&q)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = static_cast<uint32_t>(__builtin_amdgcn_fmed3f(__builtin_rintf(x[j] * s.inv) + s.zero, 0.0f, 15.0f));
}
template <bool BF16>
__device__ __forceinline__ void codes4(u4 v, const Scaling4& s, uint32_t (&q)[8]) {
  float x[8];
  widen8<BF16>(v, x);
  codes4(x, s, q);
}
__device__ __forceinline__ uint32_t pack4(const uint32_t (&q)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= q[j] << (4 * j);
  return w;
}

// What the page holds that a new token's codes depend on, read early: the scale, or the
// words that get the token's codes of v.
__device__ __forceinline__ float held_of(const KvPool& pool, int64_t ph, int slot, int team, bool there) {
  return there && slot > 0 && team < 2 ? (team == 1 ? pool.v_scale : pool.k_scale)[ph] : 0.0f;
}
struct HeldWords {
  u4 a, b;
};
__device__ __forceinline__ HeldWords held_of(const KvPool4& pool, int64_t ph, int slot, int team, bool there) {
  HeldWords h{u4{0, 0, 0, 0}, u4{0, 0, 0, 0}};
  if (there && team == 1) {
    const int c = threadIdx.x & (pool.dim / 8 - 1);
    const u4* p = reinterpret_cast<const u4*>(pool.v + (ph * (pool.block / kGroup) + slot / kGroup) * pool.dim + c * 8);
    h.a = p[0];
    h.b = p[1];
  }
  return h;
}

// Eight codes, one a byte, as a word (slots without a new row hold anything).
__device__ __forceinline__ uint32_t squeeze4(uint2 b) {
  const auto squeeze = [](uint32_t y) {
    y &= 0x0F0F0F0Fu;
    y = (y | (y >> 4)) & 0x00FF00FFu;
    return (y | (y >> 8)) & 0xFFFFu;
  };
  return squeeze(b.x) | (squeeze(b.y) << 16);
}

// The older codes of k and v of a (page, head) at a larger scale, by the whole workgroup:
// codes from `slot` on stay.  Four pieces of 16 codes a thread are on their way at a time.
// (64 sequences of 8 kv heads, all scales growing, over the same call at fixed scales: a
// full page of 128 tokens 11.0 us, with one wave and a piece at a time 12.5; of 64 tokens
// 5.5 and 5.8.)
__device__ __forceinline__ void rescale_older(int8_t* k, int8_t* v, int dim, int b, int slot, float k_ratio, float v_ratio) {
  constexpr int kAhead = 4;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int k_pieces = k_ratio != 1.0f ? slot * dim / 16 : 0;
  const int row_pieces = (slot + 15) / 16, all = k_pieces + (v_ratio != 1.0f ? dim * row_pieces : 0);  // k's, then v's
  const auto at = [&](int u, int& older) {
    if (u < k_pieces) {
      older = 16;
      return reinterpret_cast<u4*>(k) + u;
    }
    const int r = (u - k_pieces) / row_pieces, g = u - k_pieces - r * row_pieces;
    older = slot - g * 16;
    return reinterpret_cast<u4*>(v + r * b + g * 16);
  };
  for (int u0 = tid; u0 < all; u0 += threads * kAhead) {
    u4 old[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      int older;
      if (u0 + e * threads < all) old[e] = *at(u0 + e * threads, older);
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int u = u0 + e * threads;
      if (u >= all) break;
      int older;
      u4* p = at(u, older);
      const float ratio = u < k_pieces ? k_ratio : v_ratio;
      const uint32_t ow[4] = {old[e].x, old[e].y, old[e].z, old[e].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(max(older - 4 * i, 0), 4);
        const uint32_t keep = n == 4 ? 0u : ~0u << (8 * n);
        o[i] = (rescale4(ow[i], ratio) & ~keep) | (ow[i] & keep);
      }
      *p = u4{o[0], o[1], o[2], o[3]};
    }
  }
}

// One new token's key and value of a head into the page's `slot`, by a workgroup that knows
// the page: lanes of team 0 hold k, those of team 1 v.
template <bool BF16>
__device__ __forceinline__ void put_one(const KvPool& pool, int64_t ph, int slot, int team, int c, u4 raw, float was) {
  __shared__ float ratios[2];
  const int dim = pool.dim, b = pool.block, lanes = dim / 8;
  const bool is_v = team == 1, mine = team < 2;
  int8_t* k = pool.k + ph * dim * b;
  int8_t* v = pool.v + ph * dim * b;
  Scaling s{};
  if (threadIdx.x < 64) {
    s = scaling(was, group_max(mine ? absmax8<BF16>(raw) : 0.0f, lanes));
    if (mine && c == 0) ratios[team] = s.ratio;
  }
  if (slot > 0) {
    __syncthreads();
    rescale_older(k, v, dim, b, slot, ratios[0], ratios[1]);
    __syncthreads();  // a new code of v may lie in a piece stored there
  }
  float* scale_at = (is_v ? pool.v_scale : pool.k_scale) + ph;
  if (!mine) return;
  if (c == 0) *scale_at = s.now;
  int q[8];
  quant8<BF16>(raw, s.inv, q);
  if (!is_v) {
    *reinterpret_cast<uint2*>(k + static_cast<int64_t>(slot) * dim + c * 8) =
        uint2{pack_i8x4(q[0], q[1], q[2], q[3]), pack_i8x4(q[4], q[5], q[6], q[7])};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[static_cast<int64_t>(c * 8 + e) * b + slot] = static_cast<int8_t>(q[e]);
  }
}
template <bool BF16>
__device__ __forceinline__ void put_one(const KvPool4& pool, int64_t ph, int slot, int team, int c, u4 raw, const HeldWords& held) {
  const int dim = pool.dim, b = pool.block;
  if (threadIdx.x >= 64) return;
  const Scaling4 s = scaling4_of<BF16>(raw, dim / 8);
  if (team >= 2) return;
  uint32_t q[8];
  codes4<BF16>(raw, s, q);
  const int64_t row = ph * b + slot;
  if (c == 0) (team == 1 ? pool.v_scale : pool.k_scale)[row] = s.word;
  if (team == 0) {
    pool.k[row * (dim / 8) + c] = pack4(q);
    return;
  }
  u4* p = reinterpret_cast<u4*>(pool.v + (ph * (b / kGroup) + slot / kGroup) * dim + c * 8);
  const int at = 4 * (slot % kGroup);
  const uint32_t keep = ~(15u << at);
  const u4 a = held.a, d = held.b;
  p[0] = u4{(a.x & keep) | (q[0] << at), (a.y & keep) | (q[1] << at), (a.z & keep) | (q[2] << at), (a.w & keep) | (q[3] << at)};
  p[1] = u4{(d.x & keep) | (q[4] << at), (d.y & keep) | (q[5] << at), (d.z & keep) | (q[6] << at), (d.w & keep) | (q[7] << at)};
}

// A group of 8 neighbouring places of a sequence (the first a multiple of 8, as the
// words of v are) that holds new rows, whether or not they have a page.
struct Unit8 {
  bool any;
  int seq, at;     // the group's first place; negative where a sequence has more new rows than tokens
  int lo, n;       // the new rows' first slot of the group, and how many
  int64_t row;     // of q, k and v: the first of them
};
template <typename Args>
__device__ Unit8 find_unit(const Args& a, int unit) {
  Unit8 r{};
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const int s = s0 + lane;
    int t0 = 0, n = 0, first = 0;
    if (s < a.seqs) {
      t0 = min(max(a.starts[s], 0), a.tokens);
      n = min(max(a.starts[s + 1], t0), a.tokens) - t0;
      first = max(a.lens[s], 0) - n;
    }
    const int count = n > 0 ? ((first + n - 1) >> 3) - (first >> 3) + 1 : 0;
    const int sum = wave_scan(count);
    const unsigned long long hit = __ballot(before + sum > unit);
    if (hit != 0) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      const int nth = unit - before - (__builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(count, src));
      t0 = __builtin_amdgcn_readlane(t0, src);
      n = __builtin_amdgcn_readlane(n, src);
      first = __builtin_amdgcn_readlane(first, src);
      r.any = true;
      r.seq = s0 + src;
      r.at = ((first >> 3) + nth) * kGroup;
      r.lo = max(first - r.at, 0);
      r.n = min(first + n - r.at, kGroup) - r.lo;
      r.row = t0 + (r.at + r.lo - first);
      return r;
    }
    before += last_lane(sum);
  }
  return r;
}

// Each slot's turns of a group.
template <typename Args>
__device__ __forceinline__ void fill_turns(const Args& a, const Unit8& w, Turn* turns) {
  const int half = a.turn.rot / 2;
  for (int i = threadIdx.x; i < w.n * half; i += blockDim.x) {
    const int r = i / half, p = i - r * half;
    turns[(w.lo + r) * half + p] = turn_of(a.turn, p, w.row + r, w.at + w.lo + r);
  }
}

// The query heads of a group's rows, turned.
template <bool BF16, typename Args>
__device__ __forceinline__ void turn_queries(const Args& a, const Unit8& w, const Turner<kAnyRows>& t) {
  const int log2 = a.pool.dim == 64 ? 3 : 4, c = threadIdx.x & ((1 << log2) - 1), slot = (threadIdx.x >> log2) & 7;
  const int step = blockDim.x >> (log2 + 3);
  const bool mine = slot >= w.lo && slot < w.lo + w.n;
  const int64_t row = w.row + slot - w.lo;
  constexpr int kAhead = 4;
  for (int g0 = 0; g0 < a.q.heads; g0 += step * kAhead) {
    Piece p[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int h = g0 + e * step + (threadIdx.x >> (log2 + 3));
      p[e] = Piece{};
      if (mine && h < a.q.heads) p[e] = t.load(a.q.in + row * a.q.in_token + h * a.q.in_head, c, a.q_wide);
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int h = g0 + e * step + (threadIdx.x >> (log2 + 3));
      const u4 y = t.finish<BF16>(p[e], mine ? slot : w.lo, c, 0);
      if (mine && h < a.q.heads) store16(a.q.out + row * a.q.out_token + h * a.q.out_head + c * 8, y, a.q_wide);
    }
  }
}

// Codes of v of a block of heads for a group's 8 places, one a byte: a place's bytes lie
// 8 apart in a value's row, heads 1088 bytes apart (lanes then meet different banks).
constexpr int kTileHead = 1088;

// Rows that are 16-byte aligned, rot a multiple of 16: a wave takes a row, a lane 16
// values of a head, and the row's heads (of q, and for 4 bits of k and v) go by in blocks
// of a wave's lanes, neighbours in memory, the next block's values ahead.  A lane's place
// in its heads stays, and with it its turns.  Blocks [first, last) of the row; KV: 8
// waves, whose codes of v meet in `tile`.
template <int DIM, bool BF16, bool INTER, bool KV, typename Args>
__device__ __forceinline__ void append_group(const Args& a, const Unit8& w, Turn* turns, uint8_t* tile, int first, int last) {
  constexpr int kLog2 = DIM == 64 ? 2 : 3, kLanes = 1 << kLog2, kHeads = 64 / kLanes;  // lanes of a head, heads of a block
  const int half = a.turn.rot / 2, hk = a.pool.kv_heads, lane = threadIdx.x & 63, wave = static_cast<int>(threadIdx.x) >> 6;
  const int waves = static_cast<int>(blockDim.x) >> 6, c = lane & (kLanes - 1), sub = lane >> kLog2;
  const HeadLane turned = head_lane<INTER>(c, DIM / 16, a.turn.rot);
  // small loads first
  const int all_turns = w.n * half;
  const auto input = [&](int i) {
    const int r = i / half;
    return turn_input(a.turn, i - r * half, w.row + r, w.at + w.lo + r);
  };
  TurnInput mine_turn{0, 0.0f};
  if (static_cast<int>(threadIdx.x) < all_turns) mine_turn = input(threadIdx.x);
  int page = -1;
  if (KV && w.at >= 0 && w.at / a.pool.block < a.width) page = a.table[static_cast<int64_t>(w.seq) * a.table_stride + w.at / a.pool.block];
  struct Head {
    int side, head;  // 3: none
    int lo, hi;      // its pieces (v's are neighbours)
  };
  const auto head_of = [&](int block) {
    Head h{0, block * kHeads + sub, turned.lo, turned.hi};
    if (h.head >= a.q.heads) h.head -= a.q.heads, h.side = 1;
    if (h.side == 1 && h.head >= hk) h.head -= hk, h.side = 2;
    if (block >= last || (h.side > 0 && !KV) || (h.side == 2 && h.head >= hk)) h.side = 3;
    if (h.side == 2) h.lo = 16 * c, h.hi = 16 * c + 8;
    return h;
  };
  u4 lo, hi;
  const auto load = [&](const Head& h, int64_t row) {
    lo = hi = u4{0, 0, 0, 0};
    if (h.side == 3) return;
    const uint16_t* in = h.side == 0 ? a.q.in + row * a.q.in_token + h.head * a.q.in_head
                                     : h.side == 1 ? a.k + row * a.k_token + h.head * a.k_head : a.v + row * a.v_token + h.head * a.v_head;
    lo = *reinterpret_cast<const u4*>(in + h.lo);
    hi = *reinterpret_cast<const u4*>(in + h.hi);
  };
  // the wave's first row, of the group's n (KV: it has one or none)
  int r = wave;
  Head now = head_of(first);
  lo = hi = u4{0, 0, 0, 0};
  if (r < w.n) load(now, w.row + r);
  if (static_cast<int>(threadIdx.x) < all_turns) turns[threadIdx.x] = mine_turn.turn();
  for (int i = threadIdx.x + blockDim.x; i < all_turns; i += blockDim.x) turns[i] = input(i).turn();
  __syncthreads();
  const bool norms = a.turn.weight[0] != nullptr || a.turn.weight[1] != nullptr;
  const bool there = KV && page >= 0 && page < a.pool.blocks;
  const int place = w.at & (a.pool.block - 1);  // the group's in the page
  float wx[8], wz[8];
  int weight_side = -1;
  for (int block = first; KV ? block < last : r < w.n;) {
    const bool real = r < w.n;
    const Turn* t = turns + (real ? r : 0) * half;
    float x[8], z[8];
    widen8<BF16>(lo, x);
    widen8<BF16>(hi, z);
    const Head h = now;
    const int64_t row = w.row + r;
    const int slot = w.lo + r;
    const int this_block = block++;
    if (!KV && block == last) block = first, r += waves;
    now = head_of(block);
    if (r < w.n && block < last) load(now, w.row + r);
    if (real) {
      if (norms && __any(h.side < 2)) {
        const float inv = inverse_norm(group_sum(squares(x) + squares(z), kLanes), a.turn.inv_dim, a.turn.eps);
        if (h.side < 2 && side_weight(a.turn, h.side) != nullptr) {
          if (weight_side != h.side) {
            weights8<BF16>(a.turn, h.side, h.lo, wx);
            weights8<BF16>(a.turn, h.side, h.hi, wz);
            weight_side = h.side;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = normed(x[i], inv, wx[i]);
            z[i] = normed(z[i], inv, wz[i]);
          }
        }
      }
      if (h.side < 2) turn16<INTER>(x, z, turned, t);
      const u4 xb = round8<BF16>(x), zb = round8<BF16>(z);
      if (h.side == 0) {
        uint16_t* out = a.q.out + row * a.q.out_token + h.head * a.q.out_head;
        *reinterpret_cast<u4*>(out + h.lo) = xb;
        *reinterpret_cast<u4*>(out + h.hi) = zb;
      }
      if (KV && there && __any(h.side == 1 || h.side == 2)) {
        // what is held is what the storage type has (v's values are, as they came)
        widen8<BF16>(xb, x);
        widen8<BF16>(zb, z);
        float least = 0.0f, most = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          least = fminf(least, fminf(x[i], z[i]));
          most = fmaxf(most, fmaxf(x[i], z[i]));
        }
        const Scaling4 sc = scaling4(-group_max(-least, kLanes), group_max(most, kLanes));
        uint32_t q[8], p[8];
        codes4(x, sc, q);
        codes4(z, sc, p);
        const int64_t token = (static_cast<int64_t>(page) * hk + h.head) * a.pool.block + place + slot;
        if (c == 0 && (h.side == 1 || h.side == 2)) (h.side == 2 ? a.pool.v_scale : a.pool.k_scale)[token] = sc.word;
        if (h.side == 1) {
          uint32_t* k = reinterpret_cast<uint32_t*>(a.pool.k) + token * (DIM / 8);
          k[h.lo / 8] = pack4(q);
          k[h.hi / 8] = pack4(p);
        } else if (h.side == 2) {
          uint8_t* at = tile + sub * kTileHead + c * 8 + slot;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            at[i * kLanes * 8] = static_cast<uint8_t>(q[i]);
            at[(8 + i) * kLanes * 8] = static_cast<uint8_t>(p[i]);
          }
        }
      }
    }
    if constexpr (KV) {
      // (which heads a block has is the same in the whole workgroup)
      const int v0 = a.q.heads + hk;
      if (!there || (this_block + 1) * kHeads <= v0) continue;
      __syncthreads();
      const uint32_t fresh = (w.n == kGroup ? ~0u : (1u << (4 * w.n)) - 1u) << (4 * w.lo);
      for (int u = threadIdx.x; u < kHeads * DIM; u += blockDim.x) {
        const int s = u / DIM, d = u % DIM, head = this_block * kHeads + s - v0;
        if (head < 0 || head >= hk) continue;
        const uint2 b = *reinterpret_cast<const uint2*>(tile + s * kTileHead + ((d & 15) * kLanes + (d >> 4)) * 8);
        const uint32_t code = squeeze4(b);
        uint32_t* v = reinterpret_cast<uint32_t*>(a.pool.v) +
                      ((static_cast<int64_t>(page) * hk + head) * (a.pool.block / kGroup) + place / kGroup) * DIM + d;
        *v = w.n == kGroup ? code : (*v & ~fresh) | (code & fresh);
      }
      __syncthreads();
    }
  }
}

// Keys of a page, turned.
template <bool BF16, int MODE>
struct TurnedKeys {
  typedef Piece Raw;
  Turner<MODE> t;
  int rows;
  bool wide;
  __device__ __forceinline__ Piece load(const uint16_t* row, int c) const { return t.load(row, c, wide); }
  __device__ __forceinline__ u4 finish(const Piece& raw, int row, int c) const {
    const u4 y = t.template finish<BF16>(raw, row < rows ? row : 0, c, 1);
    return row < rows ? y : u4{0, 0, 0, 0};
  }
};

}  // namespace

// One new token a sequence: one workgroup holds a (sequence, kv head), its key in the
// first dim / 8 lanes, its value in the next, its query heads behind them.
template <bool BF16, int MODE, typename Args>
__global__ __launch_bounds__(kOneThreads) void rope_append_one_kernel(Args a) {
  __shared__ Turn turns[kMaxHead / 2];
  __shared__ float weights[2][kMaxHead];
  const int seq = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, dim = a.pool.dim, b = a.pool.block;
  const int log2 = dim == 64 ? 3 : 4, teams = static_cast<int>(blockDim.x) >> log2, team = tid >> log2, c = tid & ((1 << log2) - 1);
  const int pos = max(a.lens[seq], 0) - 1, half = a.turn.rot / 2, group = a.q.heads / a.pool.kv_heads;
  const bool has_place = pos >= 0 && pos < a.width * b;
  const int page = has_place ? a.table[static_cast<int64_t>(seq) * a.table_stride + pos / b] : -1;
  const Turner<MODE> t{&a.turn, turns, weights, dim, half};
  const uint16_t* q = a.q.in + seq * a.q.in_token;
  // small loads first: loads are answered in order
  TurnInput mine{0, 0.0f};
  if (tid < half) mine = turn_input(a.turn, tid, seq, pos);
  float weight[2][kMaxHead / 64];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < kMaxHead / 64; ++i) {
      weight[s][i] = 0.0f;
      if (a.turn.weight[s] != nullptr && tid < 64 && tid + 64 * i < dim) weight[s][i] = weight_at<BF16>(a.turn, s, tid + 64 * i);
    }
  // the heads' pieces: k, v, then queries
  Piece own{};
  if (team == 0) own = t.load(a.k + seq * a.k_token + head * a.k_head, c, a.wide);
  if (team == 1) own.own = load16(a.v + seq * a.v_token + head * a.v_head + c * 8, a.wide);
  if (team >= 2 && team - 2 < group) own = t.load(q + (head * group + team - 2) * a.q.in_head, c, a.q_wide);
  const bool there = page >= 0 && page < a.pool.blocks;  // else the token has no place
  const int64_t ph = static_cast<int64_t>(there ? page : 0) * a.pool.kv_heads + head;
  const auto held = held_of(a.pool, ph, pos % b, team, there);
  if (tid < half) turns[tid] = mine.turn();
  if (tid < 64)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < kMaxHead / 64; ++i) weights[s][tid + 64 * i] = weight[s][i];
  __syncthreads();
  const auto put_query = [&](int g, u4 y) {
    store16(a.q.out + seq * a.q.out_token + (head * group + g) * a.q.out_head + c * 8, y, a.q_wide);
  };
  u4 y = t.template finish<BF16>(own, 0, c, team == 0 ? 1 : 0);
  if (team >= 2 && team - 2 < group) put_query(team - 2, y);
  for (int g0 = teams - 2; g0 < group; g0 += teams) {
    const int g = g0 + team;
    Piece p{};
    if (g < group) p = t.load(q + (head * group + g) * a.q.in_head, c, a.q_wide);
    const u4 z = t.template finish<BF16>(p, 0, c, 0);
    if (g < group) put_query(g, z);
  }
  if (!there) return;
  if (team == 1) y = own.own;
  put_one<BF16>(a.pool, ph, pos % b, team, c, y, held);
}

// 8 bits, any number of new tokens: one workgroup holds one touched (page, kv head)
// as in the plain append; behind those, one turns the queries of a group of 8 rows.
template <bool BF16, int MODE, int kPer, int kThreads>
__global__ __launch_bounds__(kThreads) void rope_append_pages_kernel(RopeAppendArgs a) {
  extern __shared__ __align__(16) int8_t tile[];  // v: [dim][block] codes of the new tokens; then the turns
  __shared__ float weights[2][kMaxHead];
  const int dim = a.pool.dim, half = a.turn.rot / 2;
  const int64_t page_units = static_cast<int64_t>(a.pages) * a.pool.kv_heads;
  Turn* turns = reinterpret_cast<Turn*>(tile + dim * a.pool.block);
  const Turner<MODE> t{&a.turn, turns, weights, dim, half};
  if (blockIdx.x >= page_units) {
    const int index = static_cast<int>(blockIdx.x - page_units), unit = index / a.q_blocks;
    const Unit8 w = find_unit(a, unit);
    if (!w.any) return;
    if constexpr (MODE != kAnyRows) {
      const int first = (index - unit * a.q_blocks) * a.q_units, last = min(first + a.q_units, a.q_all);
      if (dim == 64) append_group<64, BF16, MODE == kPairs, false>(a, w, turns, nullptr, first, last);
      else append_group<128, BF16, MODE == kPairs, false>(a, w, turns, nullptr, first, last);
    } else {
      fill_weights<BF16>(a.turn, dim, weights);
      fill_turns(a, w, turns);
      __syncthreads();
      turn_queries<BF16>(a, w, t);
    }
    return;
  }
  const int unit = static_cast<int>(blockIdx.x / a.pool.kv_heads), head = static_cast<int>(blockIdx.x - static_cast<int64_t>(unit) * a.pool.kv_heads);
  const Touched w = find_block(a, unit);
  if (!w.any) return;
  const int page = a.table[static_cast<int64_t>(w.seq) * a.table_stride + w.j];
  if (page < 0 || page >= a.pool.blocks) return;  // no such page: the tokens have no place
  const int n = w.hi - w.lo;
  fill_weights<BF16>(a.turn, dim, weights);
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int r = i / half;
    turns[i] = turn_of(a.turn, i - r * half, w.token + r, w.lo + r);
  }
  __syncthreads();
  append_page<BF16, kPer, kThreads>(a, w, page, head, tile, TurnedKeys<BF16, MODE>{t, n, a.wide});
}

// 4 bits, any number of new tokens: one workgroup holds a group of 8 neighbouring
// places of a sequence, whose codes of v share words.
template <bool BF16>
__global__ __launch_bounds__(256) void rope_append4_kernel(RopeAppend4Args a) {
  constexpr int kBatch = 1024;  // values of a place whose codes meet in LDS at a time
  __shared__ Turn turns[kGroup * kMaxHead / 2];
  __shared__ float weights[2][kMaxHead];
  __shared__ __align__(8) uint8_t tile[kBatch * kGroup];
  const Unit8 w = find_unit(a, blockIdx.x);
  if (!w.any) return;
  const int dim = a.pool.dim, b = a.pool.block, hk = a.pool.kv_heads, half = a.turn.rot / 2, tid = threadIdx.x;
  const int log2 = dim == 64 ? 3 : 4, c = tid & ((1 << log2) - 1), slot = (tid >> log2) & 7, step = 256 >> (log2 + 3);
  const Turner<kAnyRows> t{&a.turn, turns, weights, dim, half};
  fill_weights<BF16>(a.turn, dim, weights);
  fill_turns(a, w, turns);
  __syncthreads();
  int page = -1;
  if (w.at >= 0 && w.at / b < a.width) page = a.table[static_cast<int64_t>(w.seq) * a.table_stride + w.at / b];
  if (page >= 0 && page < a.pool.blocks) {
    const bool mine = slot >= w.lo && slot < w.lo + w.n;
    const int64_t row = w.row + slot - w.lo;
    const int first = w.at % b;  // the group's place in the page
    const int batch = kBatch / dim;
    for (int b0 = 0; b0 < hk; b0 += batch) {
      const int b1 = min(b0 + batch, hk);
      for (int g0 = b0; g0 < b1; g0 += step) {
        const int h = g0 + (tid >> (log2 + 3));
        const bool real = mine && h < b1;
        Piece k{};
        u4 v = u4{0, 0, 0, 0};
        if (real) {
          k = t.load(a.k + row * a.k_token + h * a.k_head, c, a.wide);
          v = load16(a.v + row * a.v_token + h * a.v_head + c * 8, a.wide);
        }
        const u4 y = t.template finish<BF16>(k, mine ? slot : w.lo, c, 1);
        const Scaling4 ks = scaling4_of<BF16>(y, dim / 8), vs = scaling4_of<BF16>(v, dim / 8);
        if (!real) continue;
        const int64_t at = (static_cast<int64_t>(page) * hk + h) * b + first + slot;
        uint32_t q[8];
        codes4<BF16>(y, ks, q);
        a.pool.k[at * (dim / 8) + c] = pack4(q);
        if (c == 0) {
          a.pool.k_scale[at] = ks.word;
          a.pool.v_scale[at] = vs.word;
        }
        codes4<BF16>(v, vs, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[((h - b0) * dim + c * 8 + j) * kGroup + slot] = static_cast<uint8_t>(q[j]);
      }
      __syncthreads();
      const uint32_t fresh = (w.n == kGroup ? ~0u : (1u << (4 * w.n)) - 1u) << (4 * w.lo);
      for (int u = tid; u < (b1 - b0) * dim; u += 256) {
        const uint2 x = *reinterpret_cast<const uint2*>(tile + u * kGroup);
        const uint32_t code = squeeze4(x);
        const int h = b0 + u / dim, d = u % dim;
        uint32_t* p = a.pool.v + ((static_cast<int64_t>(page) * hk + h) * (b / kGroup) + first / kGroup) * dim + d;
        *p = w.n == kGroup ? code : (*p & ~fresh) | (code & fresh);
      }
      if (b1 < hk) __syncthreads();
    }
  }
  turn_queries<BF16>(a, w, t);
}

// The same on rows that are 16-byte aligned with rot a multiple of 16.
template <int DIM, bool BF16, bool INTER>
__global__ __launch_bounds__(kGroupThreads) void rope_append4_wide_kernel(RopeAppend4Args a) {
  __shared__ Turn turns[kGroup * DIM / 2];
  __shared__ __align__(8) uint8_t tile[1024 / DIM * kTileHead];
  const Unit8 w = find_unit(a, blockIdx.x);
  if (!w.any) return;
  const int first = static_cast<int>(blockIdx.y) * a.q_units;
  append_group<DIM, BF16, INTER, true>(a, w, turns, tile, first, min(first + a.q_units, a.q_all));
}

namespace {

template <typename Args>
int mode_of(const Args& a) {
  if (!a.wide || (a.q.heads > 0 && !a.q_wide) || a.turn.rot % 16 != 0) return kAnyRows;
  return a.turn.interleaved ? kPairs : kHalves;
}

template <int MODE, typename Args>
hipError_t launch_one_of(const Args& a) {
  const dim3 grid(static_cast<unsigned>(a.seqs), static_cast<unsigned>(a.pool.kv_heads));
  // waves for all of a kv head's query heads, up to kOneThreads
  const int lanes = (2 + a.q.heads / a.pool.kv_heads) * (a.pool.dim / 8), threads = lanes < kOneThreads ? (lanes + 63) / 64 * 64 : kOneThreads;
  if (!grid_fits(a.seqs, threads)) return kTooLarge;
  if (a.bf16) hipLaunchKernelGGL((rope_append_one_kernel<true, MODE, Args>), grid, dim3(threads), 0, a.stream, a);
  else hipLaunchKernelGGL((rope_append_one_kernel<false, MODE, Args>), grid, dim3(threads), 0, a.stream, a);
  return hipGetLastError();
}
template <typename Args>
hipError_t launch_one(const Args& a) {
  const int mode = mode_of(a);
  return mode == kHalves ? launch_one_of<kHalves>(a) : mode == kPairs ? launch_one_of<kPairs>(a) : launch_one_of<kAnyRows>(a);
}

// Blocks of heads that a workgroup takes of `all`: all of them where the call has many
// groups, else fewer, so that several workgroups share a group.  (Two sequences of 128-value
// heads, 63 MB: 15.6 us with this many workgroups, 19.4 with twice, 20.5 with four times;
// five, 224 MB: 53 us, with 8 times as many 66.)
constexpr int kWorkgroups = 512;
int units_of(int all, int64_t groups) {
  const int64_t each = all * groups / kWorkgroups;
  return static_cast<int>(each < 1 ? 1 : each < all ? each : all);
}
template <int DIM, bool INTER>
void launch_wide(const RopeAppend4Args& a, dim3 grid, dim3 block) {
  if (a.bf16) hipLaunchKernelGGL((rope_append4_wide_kernel<DIM, true, INTER>), grid, block, 0, a.stream, a);
  else hipLaunchKernelGGL((rope_append4_wide_kernel<DIM, false, INTER>), grid, block, 0, a.stream, a);
}

template <int MODE, int PER, int THREADS>
hipError_t launch_pages_of(RopeAppendArgs a) {
  // workgroups of a group's query heads
  a.q_all = (a.q.heads * (a.pool.dim / 16) + 63) / 64;
  a.q_units = MODE != kAnyRows ? units_of(a.q_all, a.units) : a.q_all;
  a.q_blocks = a.q_all > 0 ? (a.q_all + a.q_units - 1) / a.q_units : 1;
  const int64_t grid = static_cast<int64_t>(a.pages) * a.pool.kv_heads + static_cast<int64_t>(a.units) * a.q_blocks;
  if (!grid_fits(grid, THREADS)) return kTooLarge;
  const size_t rows = a.pool.block > kGroup ? a.pool.block : kGroup;
  const size_t lds = static_cast<size_t>(a.pool.dim) * a.pool.block + rows * (a.turn.rot / 2) * sizeof(Turn);
  const auto kernel = a.bf16 ? rope_append_pages_kernel<true, MODE, PER, THREADS> : rope_append_pages_kernel<false, MODE, PER, THREADS>;
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(THREADS), lds, a.stream, a);
  return hipGetLastError();
}
template <int PER, int THREADS>
hipError_t launch_pages(const RopeAppendArgs& a) {
  const int mode = mode_of(a);
  return mode == kHalves ? launch_pages_of<kHalves, PER, THREADS>(a)
                         : mode == kPairs ? launch_pages_of<kPairs, PER, THREADS>(a) : launch_pages_of<kAnyRows, PER, THREADS>(a);
}

// Groups of 8 places with new rows, at most.
template <typename Args>
int64_t most_units(const Args& a) { return a.tokens / kGroup + 2 * static_cast<int64_t>(a.seqs); }

}  // namespace

hipError_t launch_rope_append(const RopeAppendArgs& given) {
  if (given.starts == nullptr) return launch_one(given);
  RopeAppendArgs a = given;
  const int64_t pages = a.tokens / a.pool.block + 2 * static_cast<int64_t>(a.seqs);
  if (!grid_fits(pages, 256) || !grid_fits(most_units(a), 256)) return kTooLarge;  // (and both are within an int)
  a.pages = static_cast<int>(pages);
  a.units = a.q.heads > 0 ? static_cast<int>(most_units(a)) : 0;
  switch (a.pool.dim * a.pool.block / 2048) {
    case 8: return launch_pages<4, 512>(a);
    case 4: return launch_pages<4, 256>(a);
    case 2: return launch_pages<2, 256>(a);
    default: return launch_pages<1, 256>(a);
  }
}

hipError_t launch_rope_append4(const RopeAppend4Args& given) {
  if (given.starts == nullptr) return launch_one(given);
  RopeAppend4Args a = given;
  if (!grid_fits(most_units(a), mode_of(a) != kAnyRows ? kGroupThreads : 256)) return kTooLarge;
  a.units = static_cast<int>(most_units(a));
  if (mode_of(a) != kAnyRows) {
    a.q_all = ((a.q.heads + 2 * a.pool.kv_heads) * (a.pool.dim / 16) + 63) / 64;
    a.q_units = units_of(a.q_all, a.units);
    const dim3 grid(static_cast<unsigned>(a.units), static_cast<unsigned>((a.q_all + a.q_units - 1) / a.q_units)), block(kGroupThreads);
    if (a.pool.dim == 64) {
      if (a.turn.interleaved) launch_wide<64, true>(a, grid, block); else launch_wide<64, false>(a, grid, block);
    } else {
      if (a.turn.interleaved) launch_wide<128, true>(a, grid, block); else launch_wide<128, false>(a, grid, block);
    }
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(a.units));
  if (a.bf16) hipLaunchKernelGGL((rope_append4_kernel<true>), grid, dim3(256), 0, a.stream, a);
  else hipLaunchKernelGGL((rope_append4_kernel<false>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace mxq
