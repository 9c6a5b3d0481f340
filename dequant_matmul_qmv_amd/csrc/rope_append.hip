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
// Bound: HBM for prompts, launch and dependent loads for single tokens.
#include "append_device.h"
#include "turn_device.h"

namespace mxq {

namespace {

constexpr int kMaxHead = 128, kGroup = 8;  // values of a head; tokens that share a word of v
constexpr float kMaxScale4 = 4064.0f;      // 16 times it is within f16's range

// A piece of 8 values of a head, and the values they turn with.
struct Piece {
  u4 own, mate;
};

// What the turns of a workgroup's rows are made of: LDS tables of theirs and of
// the norms' weights.
struct Turner {
  const TurnArgs* turn;
  const Turn* turns;               // [rows][rot / 2]
  const float (*weights)[kMaxHead];  // of q, of k
  int dim, half;

  // Where the value that d turns with lies (itself beyond the turned part).
  __device__ __forceinline__ int mate_of(int d) const { return d < half ? d + half : d < 2 * half ? d - half : d; }
  __device__ __forceinline__ Piece load(const uint16_t* x, int c, bool wide) const {
    Piece p;
    p.own = p.mate = load16(x + c * 8, wide);
    if (!turn->interleaved && c * 8 < 2 * half) {
      if (half % 8 == 0) {
        p.mate = load16(x + mate_of(c * 8), wide);
      } else {
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
    if (turn->weight[side] != nullptr) {
      const float r = inverse_norm(group_sum(squares(x), dim / 8), turn->inv_dim, turn->eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = normed(x[j], r, weights[side][c * 8 + j]);
        z[j] = normed(z[j], r, weights[side][mate_of(c * 8 + j)]);
      }
    }
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = c * 8 + j;
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

// Largest of a head's `lanes` lanes (8 or 16).
__device__ __forceinline__ float group_max(float x, int lanes) {
  x = fmaxf(x, lane_move<0xB1, 0xF>(x));
  x = fmaxf(x, lane_move<0x4E, 0xF>(x));
  x = fmaxf(x, lane_move<0x141, 0xF>(x));
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
  const double step = (static_cast<double>(hi) - static_cast<double>(lo)) / 15.0;
  const int unit = max(__builtin_amdgcn_frexp_exp(step) - 7, -20);  // 7 bits, and f16's subnormal ones less 4
  const double up = __builtin_ldexp(__builtin_ceil(__builtin_ldexp(step, -unit)), unit);
  const float scale = fminf(static_cast<float>(up), kMaxScale4);
  Scaling4 s{0.0f, 0.0f, 0};
  if (scale > 0.0f) s.inv = static_cast<float>(1.0 / static_cast<double>(scale));
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
template <bool BF16>
__device__ __forceinline__ void codes4(u4 v, const Scaling4& s, uint32_t (&q)[8]) {
  float x[8];
  widen8<BF16>(v, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = static_cast<uint32_t>(fminf(fmaxf(__builtin_rintf(x[j] * s.inv) + s.zero, 0.0f), 15.0f));
}
__device__ __forceinline__ uint32_t pack4(const uint32_t (&q)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= q[j] << (4 * j);
  return w;
}

// One new token's key and value of a head into the page's `slot`: lanes of team 0
// hold k, those of team 1 v.
template <bool BF16>
__device__ __forceinline__ void put_one(const KvPool& pool, int64_t ph, int slot, int team, int c, u4 raw) {
  const int dim = pool.dim, b = pool.block, lane = threadIdx.x, lanes = dim / 8;
  const bool is_v = team == 1, mine = team < 2;
  float* scale_at = (is_v ? pool.v_scale : pool.k_scale) + ph;
  const float was = slot > 0 && mine ? *scale_at : 0.0f;
  const Scaling s = scaling(was, group_max(mine ? absmax8<BF16>(raw) : 0.0f, lanes));
  int8_t* k = pool.k + ph * dim * b;
  int8_t* v = pool.v + ph * dim * b;
  const float k_ratio = __shfl(s.ratio, 0), v_ratio = __shfl(s.ratio, lanes);
  if (slot > 0 && k_ratio != 1.0f)
    for (int u = lane; u < slot * dim / 16; u += 64) {
      u4* p = reinterpret_cast<u4*>(k) + u;
      const u4 o = *p;
      *p = u4{rescale4(o.x, k_ratio), rescale4(o.y, k_ratio), rescale4(o.z, k_ratio), rescale4(o.w, k_ratio)};
    }
  if (slot > 0 && v_ratio != 1.0f) {
    const int pieces = (slot + 15) / 16;  // of a row; codes from `slot` on stay
    for (int u = lane; u < dim * pieces; u += 64) {
      const int r = u / pieces, g = u - r * pieces, older = slot - g * 16;
      u4* p = reinterpret_cast<u4*>(v + static_cast<int64_t>(r) * b + g * 16);
      const u4 old = *p;
      const uint32_t ow[4] = {old.x, old.y, old.z, old.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(max(older - 4 * i, 0), 4);
        const uint32_t keep = n == 4 ? 0u : ~0u << (8 * n);
        o[i] = (rescale4(ow[i], v_ratio) & ~keep) | (ow[i] & keep);
      }
      *p = u4{o[0], o[1], o[2], o[3]};
    }
  }
  // a lane's new codes lie behind the older ones, or (v) in a piece stored above by this wave
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
__device__ __forceinline__ void put_one(const KvPool4& pool, int64_t ph, int slot, int team, int c, u4 raw) {
  const int dim = pool.dim, b = pool.block;
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
  const u4 a = p[0], d = p[1];
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

// Query heads [h0, h1) of a group's rows, turned.
template <bool BF16, typename Args>
__device__ __forceinline__ void turn_queries(const Args& a, const Unit8& w, const Turner& t, int h0, int h1) {
  const int log2 = a.pool.dim == 64 ? 3 : 4, c = threadIdx.x & ((1 << log2) - 1), slot = (threadIdx.x >> log2) & 7;
  const int step = blockDim.x >> (log2 + 3);
  const bool mine = slot >= w.lo && slot < w.lo + w.n;
  const int64_t row = w.row + slot - w.lo;
  constexpr int kAhead = 4;
  for (int g0 = h0; g0 < h1; g0 += step * kAhead) {
    Piece p[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int h = g0 + e * step + (threadIdx.x >> (log2 + 3));
      p[e] = Piece{};
      if (mine && h < h1) p[e] = t.load(a.q.in + row * a.q.in_token + h * a.q.in_head, c, a.q_wide);
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int h = g0 + e * step + (threadIdx.x >> (log2 + 3));
      const u4 y = t.finish<BF16>(p[e], mine ? slot : w.lo, c, 0);
      if (mine && h < h1) store16(a.q.out + row * a.q.out_token + h * a.q.out_head + c * 8, y, a.q_wide);
    }
  }
}

// Keys of a page, turned.
template <bool BF16>
struct TurnedKeys {
  typedef Piece Raw;
  Turner t;
  int rows;
  bool wide;
  __device__ __forceinline__ Piece load(const uint16_t* row, int c) const { return t.load(row, c, wide); }
  __device__ __forceinline__ u4 finish(const Piece& raw, int row, int c) const {
    const u4 y = t.finish<BF16>(raw, row < rows ? row : 0, c, 1);
    return row < rows ? y : u4{0, 0, 0, 0};
  }
};

}  // namespace

// One new token a sequence: one wave holds a (sequence, kv head), its key in the
// first dim / 8 lanes, its value in the next, its query heads in the others.
template <bool BF16, typename Args>
__global__ __launch_bounds__(64) void rope_append_one_kernel(Args a) {
  __shared__ Turn turns[kMaxHead / 2];
  __shared__ float weights[2][kMaxHead];
  const int seq = blockIdx.x, head = blockIdx.y, lane = threadIdx.x, dim = a.pool.dim, b = a.pool.block;
  const int log2 = dim == 64 ? 3 : 4, teams = 64 >> log2, team = lane >> log2, c = lane & ((1 << log2) - 1);
  const int pos = max(a.lens[seq], 0) - 1, half = a.turn.rot / 2, group = a.q.heads / a.pool.kv_heads;
  const Turner t{&a.turn, turns, weights, dim, half};
  const uint16_t* q = a.q.in + seq * a.q.in_token;
  // the heads' pieces: k, v, then queries
  Piece own{};
  if (team == 0) own = t.load(a.k + seq * a.k_token + head * a.k_head, c, a.wide);
  if (team == 1) own.own = load16(a.v + seq * a.v_token + head * a.v_head + c * 8, a.wide);
  if (team >= 2 && team - 2 < group) own = t.load(q + (head * group + team - 2) * a.q.in_head, c, a.q_wide);
  if (lane < half) turns[lane] = turn_of(a.turn, lane, seq, pos);
  fill_weights<BF16>(a.turn, dim, weights);
  __syncthreads();
  const auto put_query = [&](int g, u4 y) {
    store16(a.q.out + seq * a.q.out_token + (head * group + g) * a.q.out_head + c * 8, y, a.q_wide);
  };
  // (k's and q's norms are two branches: a wave goes through both)
  u4 y = t.template finish<BF16>(own, 0, c, 1);
  const u4 turned_q = t.template finish<BF16>(own, 0, c, 0);
  if (team >= 2 && team - 2 < group) put_query(team - 2, turned_q);
  for (int g0 = teams - 2; g0 < group; g0 += teams) {
    const int g = g0 + team;
    Piece p{};
    if (g < group) p = t.load(q + (head * group + g) * a.q.in_head, c, a.q_wide);
    const u4 z = t.template finish<BF16>(p, 0, c, 0);
    if (g < group) put_query(g, z);
  }
  if (pos < 0 || pos >= a.width * b) return;
  const int page = a.table[static_cast<int64_t>(seq) * a.table_stride + pos / b];
  if (page < 0 || page >= a.pool.blocks) return;  // no such page: the token has no place
  if (team == 1) y = own.own;
  put_one<BF16>(a.pool, static_cast<int64_t>(page) * a.pool.kv_heads + head, pos % b, team, c, y);
}

// 8 bits, any number of new tokens: one workgroup holds one touched (page, kv head)
// as in the plain append; behind those, one turns the queries of a group of 8 rows.
template <bool BF16, int kPer, int kThreads>
__global__ __launch_bounds__(kThreads) void rope_append_pages_kernel(RopeAppendArgs a) {
  extern __shared__ __align__(16) int8_t tile[];  // v: [dim][block] codes of the new tokens; then the turns
  __shared__ float weights[2][kMaxHead];
  const int dim = a.pool.dim, half = a.turn.rot / 2;
  const int64_t page_units = static_cast<int64_t>(a.pages) * a.pool.kv_heads;
  Turn* turns = reinterpret_cast<Turn*>(tile + dim * a.pool.block);
  const Turner t{&a.turn, turns, weights, dim, half};
  if (blockIdx.x >= page_units) {
    const Unit8 w = find_unit(a, static_cast<int>(blockIdx.x - page_units));
    if (!w.any) return;
    fill_weights<BF16>(a.turn, dim, weights);
    fill_turns(a, w, turns);
    __syncthreads();
    turn_queries<BF16>(a, w, t, 0, a.q.heads);
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
  append_page<BF16, kPer, kThreads>(a, w, page, head, tile, TurnedKeys<BF16>{t, n, a.wide});
}

// 4 bits, any number of new tokens: one workgroup holds a group of 8 neighbouring
// places of a sequence, whose codes of v share words, and a range of heads.
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
  const int each = (hk + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
  const int h0 = min(static_cast<int>(blockIdx.y) * each, hk), h1 = min(h0 + each, hk), group = a.q.heads / hk;
  const Turner t{&a.turn, turns, weights, dim, half};
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
    for (int b0 = h0; b0 < h1; b0 += batch) {
      const int b1 = min(b0 + batch, h1);
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
        const auto squeeze = [](uint32_t y) {
          y &= 0x0F0F0F0Fu;  // (slots without a new row hold anything)
          y = (y | (y >> 4)) & 0x00FF00FFu;
          return (y | (y >> 8)) & 0xFFFFu;
        };
        const uint32_t code = squeeze(x.x) | (squeeze(x.y) << 16);
        const int h = b0 + u / dim, d = u % dim;
        uint32_t* p = a.pool.v + ((static_cast<int64_t>(page) * hk + h) * (b / kGroup) + first / kGroup) * dim + d;
        *p = w.n == kGroup ? code : (*p & ~fresh) | (code & fresh);
      }
      if (b1 < h1) __syncthreads();
    }
  }
  turn_queries<BF16>(a, w, t, h0 * group, h1 * group);
}

namespace {

template <typename Args>
hipError_t launch_one(const Args& a) {
  const dim3 grid(static_cast<unsigned>(a.seqs), static_cast<unsigned>(a.pool.kv_heads));
  if (a.bf16) hipLaunchKernelGGL((rope_append_one_kernel<true, Args>), grid, dim3(64), 0, a.stream, a);
  else hipLaunchKernelGGL((rope_append_one_kernel<false, Args>), grid, dim3(64), 0, a.stream, a);
  return hipGetLastError();
}

template <int PER, int THREADS>
hipError_t launch_pages(RopeAppendArgs a) {
  const int64_t grid = static_cast<int64_t>(a.pages) * a.pool.kv_heads + a.units;
  if (!grid_fits(grid, THREADS)) return kTooLarge;
  const size_t rows = a.pool.block > kGroup ? a.pool.block : kGroup;
  const size_t lds = static_cast<size_t>(a.pool.dim) * a.pool.block + rows * (a.turn.rot / 2) * sizeof(Turn);
  const void* kernel = a.bf16 ? reinterpret_cast<const void*>(rope_append_pages_kernel<true, PER, THREADS>)
                              : reinterpret_cast<const void*>(rope_append_pages_kernel<false, PER, THREADS>);
  const hipError_t e = ensure_dynamic_lds(kernel, lds);
  if (e != hipSuccess) return e;
  const dim3 g(static_cast<unsigned>(grid));
  if (a.bf16) hipLaunchKernelGGL((rope_append_pages_kernel<true, PER, THREADS>), g, dim3(THREADS), lds, a.stream, a);
  else hipLaunchKernelGGL((rope_append_pages_kernel<false, PER, THREADS>), g, dim3(THREADS), lds, a.stream, a);
  return hipGetLastError();
}

// Groups of 8 places with new rows, at most.
template <typename Args>
int64_t most_units(const Args& a) { return a.tokens / kGroup + 2 * static_cast<int64_t>(a.seqs); }

}  // namespace

hipError_t launch_rope_append(const RopeAppendArgs& given) {
  if (given.starts == nullptr) return launch_one(given);
  RopeAppendArgs a = given;
  a.pages = static_cast<int>(a.tokens / a.pool.block + 2 * static_cast<int64_t>(a.seqs));
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
  a.units = static_cast<int>(most_units(a));
  if (!grid_fits(a.units, 256)) return kTooLarge;
  const dim3 grid(static_cast<unsigned>(a.units), 1);
  if (a.bf16) hipLaunchKernelGGL((rope_append4_kernel<true>), grid, dim3(256), 0, a.stream, a);
  else hipLaunchKernelGGL((rope_append4_kernel<false>), grid, dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace mxq
