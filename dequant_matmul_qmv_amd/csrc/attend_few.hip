// Attention of a few new tokens a sequence over the 8-bit paged cache: the
// serving step's form (one token), and short drafts.
//
//   x = (q . kcode) * kscale * scale,  p = exp(x - max x),
//   out = sum p * vscale * vcode / sum p
//
// with a key seen by a row if it is not past the row's position, inside the
// window, and its page exists; a row that sees none gives 0 and a log-sum of
// -inf.
//
// Bound: HBM, the cache read once (2 * keys * kv heads * dim bytes).  So the
// key axis is split over workgroups: every wave finds its part by a scan over
// the sequences' lengths, which only the GPU knows, and all parts are near
// equal whatever the lengths are.  The four waves of a workgroup take its
// 64-key chunks in turn and join their results in LDS; where a sequence has
// several parts, a second kernel joins those.  Measured (a copy of 1 GiB runs at
// 5.2 TB/s): two sequences of 131071 keys (537 MB) 100.6 us, 5.3 TB/s, 5 of them the
// join; 64 sequences of 5 .. 8192 keys (141 MB) 43.5 us, 3.3 TB/s, where launch, the
// search for the parts, the first loads and the join are a third; one of 777 keys 9.2 us.
//
// Both products run on the matrix cores with the codes as exact f16, straight
// from registers.  S^T = K Q^T leaves each lane 16 keys of one query row, and
// with the keys of a chunk dealt out so that those 16 are neighbours, they are
// the operand of O^T = V^T P^T as they stand: no exchange, no LDS, 16-byte
// loads of k and of v (whose tokens are innermost).  The 16 rows are the query
// heads that share a kv head, times the new tokens.
//
// Rounding: q and codes are exact, sums, maxima and weights f32; P is f16
// (2^-11 relative; the weights are summed before that rounding), held as 2^14
// times its value: normal down to 2^-28 of the row's largest.  A chunk that has
// smaller ones (rare: 19 below the largest score) multiplies them apart, in
// steps of 2^24.  v's scales differ by page: P carries vscale / the
// largest vscale so far, at most 1, and that largest one multiplies the sums.
#include <climits>

#include "attend_device.h"

namespace mxq {

namespace {

constexpr int kFewWaves = 4;    // of a workgroup; twice that where it takes all keys
constexpr int kChunk = 64;      // keys a wave takes at a time
constexpr int kLongRounds = 3;
constexpr int kMinChunks = 4;   // at least one chunk for each wave of a workgroup
// Tables of up to this many keys are not split: a workgroup of eight waves takes
// all keys of its rows, in two rounds at most.  8 kv heads, split and joined / not
// split, in us, a call among others and inside a graph (which then has no
// workspace to allocate):
//   1 sequence    64 values, 512 keys 11.3 / 8.8, 20.1 / 6.8; 1024 keys 11.3 / 8.8, 20.7 / 9.2
//                128 values, 512 keys 11.2 / 8.7, 19.5 / 8.8; 1024 keys 11.2 / 12.0, 18.7 / 12.4
//   32 sequences  64 values, 1024 keys 14.6 / 9.9, 23.0 / 10.5
//                128 values, 1024 keys 22.9 / 16.0, 31.1 / 16.8
// So 128 values, more than 512 keys and few sequences lose 1 us outside a graph
// and win 6 inside one; all others win both ways.
constexpr int kLoneKeys = 1024;
constexpr float kTiny = 1e-30f;

// One sequence's share of the few-row work.
struct Share {
  int c0, chunks;  // first 64-key chunk, and how many
  int groups;      // groups of 16 * MT rows
};
template <int MT>
__device__ __forceinline__ Share share_of(const AttendArgs& a, int s) {
  Share r{};
  if (s >= a.seqs) return r;
  const SeqSpan q = seq_span(a, s);
  const int64_t rows = static_cast<int64_t>(q.n) * a.group;
  if (rows > a.few_rows) return r;
  r.groups = static_cast<int>((rows + 16 * MT - 1) / (16 * MT));
  const int hi = min(q.len, a.width * a.pool.block);
  const int lo = first_seen(a, q.len - q.n);
  r.c0 = lo / kChunk;
  r.chunks = max(0, hi / kChunk + (hi % kChunk != 0) - r.c0);  // (hi may be near 2^31)
  return r;
}

struct Part {
  bool any;
  int seq, base, nth;   // base: the sequence's first slot; nth: the slot within it
  int step, splits;     // chunks of a part, parts of the sequence
  Share share;
};

// Where slot `slot` lies, or (slot < 0) sequence `seq`.  Run by whole waves.
template <int MT>
__device__ Part find_part(const AttendArgs& a, int slot, int seq) {
  const int lane = threadIdx.x & 63, hk = a.pool.kv_heads;
  long long total = 0;
  Share mine{};
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    mine = share_of<MT>(a, s0 + lane);
    total += static_cast<long long>(mine.chunks) * mine.groups * hk;
  }
  total = wave_sum(total);
  // Four workgroups a compute unit, or two where four would still have
  // kLongRounds chunks a wave (64 sequences up to 8192 keys: 45 us with four, 48
  // with two; 8 of 16384: 59 and 55; two of 131071: 105 and 101); parts of whole
  // rounds of the four waves (64 sequences: 48 us with parts of 9 chunks, 45 with 12).
  long long even = (total + a.target - 1) / a.target;
  if (even >= kLongRounds * kFewWaves) even *= 2;
  Part p{};
  p.step = static_cast<int>((max(even, static_cast<long long>(a.min_chunks)) + kFewWaves - 1) / kFewWaves * kFewWaves);
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    if (a.seqs > 64) mine = share_of<MT>(a, s0 + lane);
    const int splits = max(1, (mine.chunks + p.step - 1) / p.step);
    const int count = mine.groups * splits * hk;
    const int sum = wave_scan(count);
    const unsigned long long hit = slot >= 0 ? __ballot(before + sum > slot) : (seq < s0 + 64 ? 1ull << (seq - s0) : 0);
    if (hit != 0) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      p.any = true;
      p.seq = s0 + src;
      p.base = before + __builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(count, src);
      p.nth = slot - p.base;
      p.splits = __builtin_amdgcn_readlane(splits, src);
      p.share.c0 = __builtin_amdgcn_readlane(mine.c0, src);
      p.share.chunks = __builtin_amdgcn_readlane(mine.chunks, src);
      p.share.groups = __builtin_amdgcn_readlane(mine.groups, src);
      return p;
    }
    before += last_lane(sum);
  }
  return p;
}

// One lane's part of a chunk, as stored.
template <int DIM>
struct Raw {
  u4 k[4 * (DIM / 64)];
  u4 v[DIM / 16];
  float ks, vs;
  bool ok;
};

// Registers as if rewritten: what is computed from them again is not shared
// with, or kept from, an earlier computation.
__device__ __forceinline__ u4 anew(u4 w) {
  asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
  return w;
}

struct Pages {
  int k, v;   // pages of the lane's k rows and of its v tokens; -1: none
};

}  // namespace

template <int DIM, int MT, bool BF16, int WAVES>
__global__ __launch_bounds__(64 * WAVES, MT * DIM >= 256 && WAVES == kFewWaves ? 1 : 2) void attend_few_kernel(AttendArgs a) {
  constexpr int U = DIM / 64, DB = DIM / 16, kRows = 16 * MT;
  __shared__ float join[WAVES][16][DIM + 4];
  __shared__ float join_m[WAVES][16], join_l[WAVES][16], join_vs[WAVES];
  const Part part = find_part<MT>(a, blockIdx.x, -1);
  if (!part.any) return;
  const int hk = a.pool.kv_heads, block = a.pool.block;
  const int head = part.nth % hk, rest = part.nth / hk, rg = rest % part.share.groups, split = rest / part.share.groups;
  const SeqSpan sp = seq_span(a, part.seq);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rho = lane & 15, h = lane >> 4;
  const int row0 = rg * kRows, rows = min(kRows, sp.n * a.group - row0);
  const int pos0 = sp.len - sp.n;
  const int limit = min(sp.len, a.width * block);

  // query rows of this lane (one of 16 for each mt), their fragments and key ranges
  u4 qf[MT][2 * U];
  float factor[MT];
  int from[MT], upto[MT];
  int all_from = 0, all_upto = INT_MAX;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int i = row0 + mt * 16 + rho;
    const bool real = i < sp.n * a.group;
    const int tok = real ? i / a.group : 0, hq = head * a.group + (real ? i - tok * a.group : 0);
    const uint16_t* q = a.q + static_cast<int64_t>(sp.t0 + tok) * a.q_token + static_cast<int64_t>(hq) * a.q_head;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < 2; ++f) qf[mt][2 * u + f] = *reinterpret_cast<const u4*>(q + u * 64 + h * 16 + f * 8);
    float inverse = 1.0f;
    if constexpr (BF16) {
      float top = 0.0f, fac;
#pragma unroll
      for (int f = 0; f < 2 * U; ++f) top = fmaxf(top, absmax8_bf16(qf[mt][f]));
      top = max_xor16(max_xor32(top));
      row_factor(top, fac, inverse);
#pragma unroll
      for (int f = 0; f < 2 * U; ++f) qf[mt][f] = bf16_to_scaled_f16(qf[mt][f], fac);
    }
    factor[mt] = a.scale2 * inverse;
    const int pos = pos0 + tok;
    upto[mt] = min(pos + 1, limit);  // rows past the last repeat the first; they are not stored
    from[mt] = first_seen(a, pos);
    if (real) {
      all_from = max(all_from, from[mt]);
      all_upto = min(all_upto, upto[mt]);
    }
  }
  // keys that every row sees: [all_from, all_upto)
#pragma unroll
  for (int d = 1; d < 16; d *= 2) {
    all_from = max(all_from, __shfl_xor(all_from, d));
    all_upto = min(all_upto, __shfl_xor(all_upto, d));
  }

  const int32_t* table = a.table + static_cast<int64_t>(part.seq) * a.table_stride;
  const int c_begin = part.share.c0 + split * part.step;
  const int c_end = min(c_begin + part.step, part.share.c0 + part.share.chunks);
  const int kgroup = rho >> 2;  // the 16-key group whose k rows this lane loads
  const uint32_t magic = kMagic;

  auto pages_of = [&](int c) {
    Pages p;
    // (a chunk past the end may lie past 2^31)
    const uint32_t key = static_cast<uint32_t>(c) * kChunk, width = a.width;
    const uint32_t jk = (key + kgroup * 16) / block, jv = (key + h * 16) / block;
    p.k = jk < width ? table[jk] : -1;
    p.v = jv < width ? table[jv] : -1;
    return p;
  };
  auto load_k = [&](int c, Pages p, Raw<DIM>& r) {
    const int64_t pk = p.k >= 0 && p.k < static_cast<int>(a.pool.blocks) ? p.k : 0;
    const int tk = (c * kChunk + kgroup * 16) & (block - 1);
    const int8_t* kp = a.pool.k + ((pk * hk + head) * block + tk + (rho & 3)) * DIM + h * 16;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u) r.k[b * U + u] = *reinterpret_cast<const u4*>(kp + b * 4 * DIM + u * 64);
  };
  auto load_v = [&](int c, Pages p, Raw<DIM>& r) {
    // a page past the sequence's end may be anyone's, or never written
    r.ok = p.v >= 0 && p.v < static_cast<int>(a.pool.blocks) && c * kChunk + h * 16 < limit;
    const int64_t pv = r.ok ? p.v : 0;
    const int tv = (c * kChunk + h * 16) & (block - 1);
    const int8_t* vp = a.pool.v + ((pv * hk + head) * DIM + rho) * block + tv;
    r.ks = a.pool.k_scale[pv * hk + head];
    r.vs = r.ok ? a.pool.v_scale[pv * hk + head] : 0.0f;
#pragma unroll
    for (int db = 0; db < DB; ++db) r.v[db] = *reinterpret_cast<const u4*>(vp + db * 16 * block);
  };

  f4 acc[MT][DB];
  float m[MT], l[MT], top_vs = kTiny;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = kNegInf;
    l[mt] = 0.0f;
#pragma unroll
    for (int db = 0; db < DB; ++db) acc[mt][db] = f4{0, 0, 0, 0};
  }

  // one chunk: as soon as k's registers are free they take the next chunk's
  // rows, and v's do after the second product
  auto step = [&](int c, Raw<DIM>& r, Pages& ahead) {
    const bool more_chunks = c + WAVES < c_end;
    f4 s[MT][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][b] = f4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const u4 w = r.k[b * U + u];
        const h8 k0 = as_h8(codes8_f16(w.x, w.y, magic)), k1 = as_h8(codes8_f16(w.z, w.w, magic));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          s[mt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, as_h8(qf[mt][2 * u]), s[mt][b], 0, 0, 0);
          s[mt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, as_h8(qf[mt][2 * u + 1]), s[mt][b], 0, 0, 0);
        }
      }
    }
    if (more_chunks) load_k(c + WAVES, ahead, r);
    const float was_vs = top_vs;
    top_vs = fmaxf(top_vs, max_xor16(max_xor32(r.vs)));
    const float share = r.vs / top_vs, shrink = was_vs / top_vs;
    const bool whole = __all(r.ok) && c * kChunk >= all_from && c * kChunk <= all_upto - kChunk;
    const int key0 = c * kChunk + h * 16;
    bool low = false;
    float ref[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float f = r.ks * factor[mt];
      float mx = kNegInf, mn = -kNegInf;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = s[mt][i >> 2][i & 3] * f;
        if (!whole) {
          const int key = key0 + i;
          const bool seen = r.ok && key >= from[mt] && key < upto[mt];
          mn = fminf(mn, seen ? x : -kNegInf);
          x = seen ? x : kNegInf;
        } else {
          mn = fminf(mn, x);
        }
        mx = fmaxf(mx, x);
        s[mt][i >> 2][i & 3] = x;
      }
      const float now = fmaxf(m[mt], max_xor16(max_xor32(mx)));
      ref[mt] = now == kNegInf ? 0.0f : now;
      const float alpha = __builtin_amdgcn_exp2f(m[mt] - ref[mt]);
      m[mt] = now;
      l[mt] *= alpha;
      low |= __builtin_amdgcn_exp2f(mn - ref[mt] + kLift) * share < kF16Normal;
      const float down = alpha * shrink;
#pragma unroll
      for (int db = 0; db < DB; ++db) acc[mt][db] *= down;
    }
    const bool any_low = __any(low);
    u4 pf[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float sum = 0.0f;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float p0 = __builtin_amdgcn_exp2f(s[mt][i >> 2][i & 3] - ref[mt] + kLift);
        float p1 = __builtin_amdgcn_exp2f(s[mt][i >> 2][(i & 3) + 1] - ref[mt] + kLift);
        sum += p0 + p1;
        p0 *= share;
        p1 *= share;
        if (any_low) {  // kept for the second product
          s[mt][i >> 2][i & 3] = p0;
          s[mt][i >> 2][(i & 3) + 1] = p1;
          p0 = p0 < kF16Normal ? 0.0f : p0;
          p1 = p1 < kF16Normal ? 0.0f : p1;
        }
        const h2 pk = {static_cast<_Float16>(p0), static_cast<_Float16>(p1)};
        w[i / 2] = as_u32(pk);
      }
      l[mt] += sum;
      pf[mt][0] = u4{w[0], w[1], w[2], w[3]};
      pf[mt][1] = u4{w[4], w[5], w[6], w[7]};
    }
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const u4 w = r.v[db];
      const h8 v0 = as_h8(codes8_f16(w.x, w.y, magic)), v1 = as_h8(codes8_f16(w.z, w.w, magic));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        acc[mt][db] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, as_h8(pf[mt][0]), acc[mt][db], 0, 0, 0);
        acc[mt][db] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, as_h8(pf[mt][1]), acc[mt][db], 0, 0, 0);
      }
    }
    // values below f16's normal range: products of their own, until none is left
    Band band;
    for (bool more = any_low; more; band.next()) {
      bool left = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float p0 = s[mt][i >> 2][i & 3], p1 = s[mt][i >> 2][(i & 3) + 1];
          left |= band.below(p0) || band.below(p1);
          const h2 pk = {static_cast<_Float16>(band.lifted(p0)), static_cast<_Float16>(band.lifted(p1))};
          w[i / 2] = as_u32(pk);
        }
        pf[mt][0] = u4{w[0], w[1], w[2], w[3]};
        pf[mt][1] = u4{w[4], w[5], w[6], w[7]};
      }
      more = __any(left && !band.last());
#pragma unroll
      for (int db = 0; db < DB; ++db) {
        const u4 w = anew(r.v[db]);
        const h8 v0 = as_h8(codes8_f16(w.x, w.y, magic)), v1 = as_h8(codes8_f16(w.z, w.w, magic));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          f4 t = f4{0, 0, 0, 0};
          t = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, as_h8(pf[mt][0]), t, 0, 0, 0);
          t = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, as_h8(pf[mt][1]), t, 0, 0, 0);
          acc[mt][db] += t * (1.0f / band.lift);
        }
      }
    }
    if (more_chunks) {
      load_v(c + WAVES, ahead, r);
      ahead = pages_of(c + 2 * WAVES);
    }
  };

  int c = c_begin + wave;
  if (c < c_end) {
    Raw<DIM> raw;
    Pages ahead = pages_of(c);
    load_k(c, ahead, raw);
    load_v(c, ahead, raw);
    ahead = pages_of(c + WAVES);   // past the end: -1, or a page that is not used
    for (; c < c_end; c += WAVES) step(c, raw, ahead);
  }

  // join the waves, 16 rows at a time
  const bool alone = part.splits == 1;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const float weight = add_xor16(add_xor32(l[mt]));
    if (h == 0) {
      join_m[wave][rho] = m[mt];
      join_l[wave][rho] = weight;
    }
    if (lane == 0) join_vs[wave] = top_vs;
#pragma unroll
    for (int db = 0; db < DB; ++db)
      *reinterpret_cast<f4*>(&join[wave][rho][db * 16 + h * 4]) = acc[mt][db];
    __syncthreads();
    for (int u = threadIdx.x; u < 16 * (DIM / 4); u += 64 * WAVES) {
      const int row = u / (DIM / 4), d = (u - row * (DIM / 4)) * 4, i = mt * 16 + row;
      if (i < rows) {
        float top = join_m[0][row];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) top = fmaxf(top, join_m[w][row]);
        const float ref = top == kNegInf ? 0.0f : top;
        float total = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) total += join_l[w][row] * __builtin_amdgcn_exp2f(join_m[w][row] - ref);
        const float inv = over(total);
        f4 y = f4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
          y += *reinterpret_cast<const f4*>(&join[w][row][d]) * (__builtin_amdgcn_exp2f(join_m[w][row] - ref) * inv) * join_vs[w];
        if (alone) {
          const int tok = (row0 + i) / a.group, hq = head * a.group + (row0 + i) - tok * a.group;
          const int64_t at = static_cast<int64_t>(sp.t0 + tok) * a.heads + hq;
          uint16_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(y[e]);
          *reinterpret_cast<uint2*>(a.out + at * DIM + d) =
              uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                    static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
          if (a.lse && d == 0) a.lse[at] = log_sum(ref, total);
        } else {
          const int64_t at = static_cast<int64_t>(blockIdx.x) * kRows + i;
          *reinterpret_cast<f4*>(a.part + at * DIM + d) = y;
          if (d == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = float2{top, total};
        }
      }
    }
    if (mt + 1 < MT) __syncthreads();
  }
}

// One workgroup for each (token, query head): the parts of its row, 4 values a
// lane, the parts dealt over the workgroup's groups of DIM / 4 lanes.
template <int DIM, int MT, bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS) void attend_join_kernel(AttendArgs a) {
  constexpr int kLanes = DIM / 4, kTeams = THREADS / kLanes, kRows = 16 * MT;
  __shared__ float sums[kTeams][DIM];
  __shared__ float team_m[kTeams], team_l[kTeams];
  // one token a sequence, or up to `join_new`
  const int hq = blockIdx.y, seq = blockIdx.x / a.join_new, nth = blockIdx.x - seq * a.join_new;
  const SeqSpan sp = seq_span(a, seq);
  if (nth >= sp.n || static_cast<int64_t>(sp.n) * a.group > a.few_rows) return;
  const int tok = sp.t0 + nth;
  const Part part = find_part<MT>(a, -1, seq);
  if (part.splits == 1) return;
  const int hk = a.pool.kv_heads, head = hq / a.group;
  const int i = (tok - sp.t0) * a.group + hq - head * a.group, rg = i / kRows, row = i - rg * kRows;
  const int team = threadIdx.x / kLanes, d = (threadIdx.x - team * kLanes) * 4;
  float top = kNegInf, total = 0.0f;
  f4 y = f4{0, 0, 0, 0};
  // four parts at a time, so that their loads run together
  for (int s0 = team; s0 < part.splits; s0 += 4 * kTeams) {
    float2 ml[4];
    f4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = min(s0 + i * kTeams, part.splits - 1);
      // (starts that descend may give more than there are: not read)
      const int64_t slot = min(part.base + (static_cast<int64_t>(s) * part.share.groups + rg) * hk + head, static_cast<int64_t>(a.slots) - 1);
      const int64_t at = slot * kRows + row;
      ml[i] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
      v[i] = *reinterpret_cast<const f4*>(a.part + at * DIM + d);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s0 + i * kTeams >= part.splits) continue;
      const float now = fmaxf(top, ml[i].x), ref = now == kNegInf ? 0.0f : now;
      const float e0 = __builtin_amdgcn_exp2f(top - ref), w = ml[i].y * kJoinUnit * __builtin_amdgcn_exp2f(ml[i].x - ref);
      y = y * e0 + v[i] * w;
      total = total * e0 + w;
      top = now;
    }
  }
  *reinterpret_cast<f4*>(&sums[team][d]) = y;
  if (d == 0) {
    team_m[team] = top;
    team_l[team] = total;
  }
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  top = team_m[0];
#pragma unroll
  for (int t = 1; t < kTeams; ++t) top = fmaxf(top, team_m[t]);
  const float ref = top == kNegInf ? 0.0f : top;
  y = f4{0, 0, 0, 0};
  total = 0.0f;
#pragma unroll
  for (int t = 0; t < kTeams; ++t) {
    const float e = __builtin_amdgcn_exp2f(team_m[t] - ref);
    y += *reinterpret_cast<const f4*>(&sums[t][d]) * e;
    total += team_l[t] * e;
  }
  const int64_t at = static_cast<int64_t>(tok) * a.heads + hq;
  const float inv = over(total);
  uint16_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(y[e] * inv);
  *reinterpret_cast<uint2*>(a.out + at * DIM + d) = uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                                                          static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
  if (a.lse && d == 0) a.lse[at] = log_sum(ref, total / kJoinUnit);
}

namespace {

template <int DIM, int MT, int WAVES>
hipError_t launch_parts(const AttendArgs& a, unsigned slots) {
  const dim3 grid(slots), block(64 * WAVES);
  if (a.bf16) hipLaunchKernelGGL((attend_few_kernel<DIM, MT, true, WAVES>), grid, block, 0, a.stream, a);
  else hipLaunchKernelGGL((attend_few_kernel<DIM, MT, false, WAVES>), grid, block, 0, a.stream, a);
  return hipGetLastError();
}

// Waves of a workgroup: twice as many where it takes all keys of more than a
// round (32 rows of 128 values do not fit the registers of that many waves).
constexpr int lone_waves(int values) { return values >= 256 ? kFewWaves : 2 * kFewWaves; }
int few_waves(const AttendArgs& a, int values, bool joined) {
  return !joined && static_cast<int64_t>(a.width) * a.pool.block > kFewWaves * kChunk ? lone_waves(values) : kFewWaves;
}
// One wave a row joins where the sequences are too many to have many parts each
// (64 sequences: 45.4 -> 44.1 us).
int join_threads(const AttendArgs& a) { return 8 * static_cast<int64_t>(a.seqs) * a.pool.kv_heads >= a.target ? 64 : 256; }

template <int DIM, int MT>
hipError_t launch_mt(const AttendArgs& a, unsigned slots, bool joined) {
  hipError_t e = few_waves(a, MT * DIM, joined) == kFewWaves ? launch_parts<DIM, MT, kFewWaves>(a, slots)
                                                             : launch_parts<DIM, MT, lone_waves(MT * DIM)>(a, slots);
  if (e != hipSuccess || !joined) return e;
  const dim3 grid(static_cast<unsigned>(a.seqs) * static_cast<unsigned>(a.join_new), static_cast<unsigned>(a.heads));
  if (join_threads(a) == 64) {
    if (a.bf16) hipLaunchKernelGGL((attend_join_kernel<DIM, MT, true, 64>), grid, dim3(64), 0, a.stream, a);
    else hipLaunchKernelGGL((attend_join_kernel<DIM, MT, false, 64>), grid, dim3(64), 0, a.stream, a);
  } else {
    if (a.bf16) hipLaunchKernelGGL((attend_join_kernel<DIM, MT, true, 256>), grid, dim3(256), 0, a.stream, a);
    else hipLaunchKernelGGL((attend_join_kernel<DIM, MT, false, 256>), grid, dim3(256), 0, a.stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_few(const AttendArgs& a, int mt, unsigned slots, bool joined) {
  if (slots == 0) return hipSuccess;
  if (a.pool.dim == 64) return mt == 1 ? launch_mt<64, 1>(a, slots, joined) : launch_mt<64, 2>(a, slots, joined);
  return mt == 1 ? launch_mt<128, 1>(a, slots, joined) : launch_mt<128, 2>(a, slots, joined);
}

// Sequences of up to this many rows take the few-row kernel.
constexpr int kFewRows = 64;

}  // namespace

hipError_t launch_attend(const AttendArgs& given, const DeviceInfo& dev) {
  AttendArgs a = given;
  if (a.pool.blocks == 0) a.width = 0;  // no page exists: every row is empty
  const int64_t all_rows = static_cast<int64_t>(a.tokens) * a.group, hk = a.pool.kv_heads;
  // How many new tokens a sequence has is known on the GPU alone.  One kernel
  // runs where that cannot matter; else both, each with its own sequences.
  const bool few = a.starts == nullptr || a.seqs > 1 || all_rows <= kFewRows;
  const bool many = a.starts != nullptr && all_rows > kFewRows;
  a.few_rows = !many ? INT_MAX : few ? kFewRows : 0;
  a.target = dev.num_cu * 4;
  // the most new tokens of a sequence that the few-row kernel takes
  a.join_new = a.starts == nullptr ? 1 : many ? (kFewRows / a.group > 0 ? kFewRows / a.group : 1) : a.tokens;

  const int64_t most = a.starts == nullptr ? a.group : all_rows < kFewRows ? all_rows : kFewRows;
  const int mt = most <= 16 ? 1 : 2;
  // slots: at most `target` full parts, and one more for each (sequence, group of rows, kv head)
  int64_t few_total = all_rows;
  if (many && few_total > static_cast<int64_t>(a.seqs) * kFewRows) few_total = static_cast<int64_t>(a.seqs) * kFewRows;
  const int64_t per = 16 * mt, ends = few ? (few_total / per + a.seqs) * hk : 0;
  const bool joined = few && static_cast<int64_t>(a.width) * a.pool.block > kLoneKeys;
  a.min_chunks = joined ? kMinChunks : kLoneKeys / kChunk;
  const int64_t slots = ends + (joined ? a.target : 0);
  if (few && (!grid_fits(slots, 64 * few_waves(a, mt * a.pool.dim, joined)) ||
              (joined && !grid_fits(static_cast<int64_t>(a.seqs) * a.join_new, join_threads(a)))))
    return kTooLarge;
  a.slots = static_cast<int>(slots);
  const size_t sums = joined ? static_cast<size_t>(slots) * per * a.pool.dim * 4 : 0;
  const size_t few_bytes = joined ? sums + static_cast<size_t>(slots) * per * 8 : 0;

  // the many-row kernel's key axis is split while its tiles leave compute units idle
  a.many_splits = 1;
  if (many) {
    const int64_t tiles = many_tiles(a) * hk, stages = (static_cast<int64_t>(a.width) * a.pool.block + kChunk - 1) / kChunk;
    int64_t splits = tiles > 0 ? 2 * dev.num_cu / tiles : 1;
    if (splits > stages / 4) splits = stages / 4;
    if (splits > 32) splits = 32;
    if (splits > 1) a.many_splits = static_cast<int>(splits);
  }
  if (many && (!grid_fits(many_tiles(a) * hk * a.many_splits, 256) || (a.many_splits > 1 && !grid_fits(a.tokens, 256)))) return kTooLarge;
  const size_t many_bytes = many ? many_part_bytes(a) : 0;

  const auto enqueue = [&](float* ws) {
    a.part = ws;
    a.part_ml = ws + sums / 4;
    hipError_t e = many ? launch_many(a, ws + few_bytes / 4) : hipSuccess;
    if (e == hipSuccess && few) e = launch_few(a, mt, static_cast<unsigned>(slots), joined);
    return e;
  };
  if (few_bytes + many_bytes == 0) return enqueue(nullptr);
  return with_split_workspace(dev, a.stream, few_bytes + many_bytes, enqueue);
}

}  // namespace mxq
