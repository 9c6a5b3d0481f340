// Attention of a few new tokens a sequence over the 4-bit paged cache: the serving
// step's form (one token), and short drafts.
//
//   x = (q . c - z sum q) * s * scale,  p = exp(x - max x),
//   out = sum p s' (c' - z') / sum p
//
// with c, z, s a key's codes, zero point and scale, c', z', s' a value's; masks as
// for the 8-bit cache.
//
// Bound: HBM, the cache read once (keys * kv heads * (dim + 4) bytes), and beside it
// the vector ALU, which unpacks two codes where the 8-bit cache has one in the same
// byte.  The key axis is divided over workgroups as there (attend_split.h).  Measured: three
// sequences of 131000 keys of 128 values 90 us (4.6 TB/s; over 8 bits 191), 96 of up to
// 8192 keys 44 (8 bits 68).  Short parts cost their code's instruction fetches: masked
// chunks are handled without branches (one sequence of 913 keys 10.7 -> 10.2 us).
//
// Both products run on the matrix cores straight from registers.  S^T = K Q^T, keys as
// 16 rows, leaves lane group h four keys of one query row in each tile; with the rows
// of two tiles dealt out so that those are the 8 tokens that a word of v holds, in the
// order in which its codes unpack, the weights are the operand of O^T = V^T P^T in
// place.  k's codes go in as 64 + c, and a score starts from -(64 + z) sum q; its key's
// scale multiplies it afterwards.  v's go in as c - z, and their scale multiplies the
// weight.
//
// Rounding: q and codes exact (a bf16 q to 2^-25 of its row's largest); sums, maxima and
// weights f32.  P holds the weight times its value's scale over 2^k, 2^k the first power
// of two that no scale the row has seen so far reaches, in f16: normal down to 2^-27 of the
// largest.  k is a row's own: a key that it does not see costs it nothing.
#include <climits>

#include "attend4_device.h"

namespace mxq {

namespace {

// One lane's part of a chunk of 64 keys, as stored.
template <int DIM>
struct Raw4 {
  uint32_t k[4][DIM / 32];  // tiles of 16 keys; a key's values h * DIM / 4 ..
  u4 v[2][DIM / 64];        // halves of 32 keys; 4 values of 8 tokens
  u4 ks[2], vs[2];          // scale words of those 8 tokens
};

// The pages of a chunk's halves, the same in the whole wave (and of the second 16
// tokens of each half, where pages have no more); -1: none.
struct Pages4 {
  int at[2][2];
};

template <int N>
__device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u4 x = *reinterpret_cast<const u4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  }
}

__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) {
  typedef unsigned short us2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}

constexpr float kSlack4 = 1.75f;  // weights reach 2^(kLift + kSlack4), below f16's largest

}  // namespace

template <int DIM, int MT, int WAVES, bool SMALL>
__global__ __launch_bounds__(64 * WAVES, MT * DIM <= 128 ? 3 : WAVES == kFewWaves ? 1 : 2) void attend4_few_kernel(Attend4Args a) {
  constexpr int KW = DIM / 32, DP = DIM / 64, kRows = 16 * MT;
  __shared__ float join[WAVES][16][DIM + 4];
  __shared__ float join_m[WAVES][16], join_l[WAVES][16];
  // (a workgroup of more waves takes all keys of its rows: parts are one each)
  const Part part = WAVES == kFewWaves && long_first_pays(a) ? find_part_long_first<MT>(a, blockIdx.x) : find_part<MT>(a, blockIdx.x, -1);
  // (starts that descend may give more parts than there are slots: not taken)
  if (!part.any || static_cast<uint32_t>(part.base + part.nth) >= static_cast<uint32_t>(a.slots)) return;
  const int hk = a.pool.kv_heads, block = a.pool.block, block_log2 = 31 - __builtin_clz(block);
  const int head = part.nth % hk, rest = part.nth / hk, rg = rest % part.share.groups, split = rest / part.share.groups;
  const SeqSpan sp = seq_span(a, part.seq);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rho = lane & 15, h = lane >> 4;
  const int row0 = rg * kRows, rows = min(kRows, sp.n * a.group - row0);
  const int pos0 = sp.len - sp.n;
  const int limit = __builtin_amdgcn_readfirstlane(min(sp.len, a.width * block));

  const int32_t* table = a.table + static_cast<int64_t>(part.seq) * a.table_stride;
  const int c_begin = part.share.c0 + split * part.step;
  const int c_end = min(c_begin + part.step, part.share.c0 + part.share.chunks);
  // the lane's row of 32 keys in the first tile (2 further in the second), its words of k and v
  const int k_row = 8 * (rho >> 2) + 4 * (rho & 1) + ((rho >> 1) & 1);
  const uint32_t k_at = static_cast<uint32_t>(k_row * (DIM / 8) + h * KW) * 4, v_at = static_cast<uint32_t>(h * DIM + rho * 4) * 4;  // bytes

  auto pages_of = [&](int c) {
    Pages4 p;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (g == 1 && !SMALL) {
          p.at[u][1] = p.at[u][0];
          continue;
        }
        // (a chunk past the end may lie past 2^31)
        const uint32_t j = (static_cast<uint32_t>(c) * kChunk + u * 32 + g * 16) >> block_log2;
        p.at[u][g] = j < static_cast<uint32_t>(a.width) ? table[j] : -1;
      }
    return p;
  };
  Pages4 now_at;  // of the chunk at hand
  // Is the page there, and (a page past the sequence's end may be anyone's, or never written) some of its keys?
  auto there = [&](int c, const Pages4& p, int u, int g) -> bool {
    return (static_cast<uint32_t>(p.at[u][g]) < static_cast<uint32_t>(a.pool.blocks)) & (c * kChunk + u * 32 + g * 16 < limit);
  };
  // The same for the lane's 8 tokens of a half.
  auto lane_there = [&](int c, int u) -> bool {
    if constexpr (!SMALL) return there(c, now_at, u, 0);
    const bool first = there(c, now_at, u, 0), second = there(c, now_at, u, 1);
    return h >= 2 ? second : first;
  };
  // tokens before a half (or its second 16 tokens), in all of the pool's
  auto tokens_before = [&](int c, const Pages4& p, int u, int g) {
    const int64_t page = p.at[u][g] >= 0 && p.at[u][g] < static_cast<int>(a.pool.blocks) ? p.at[u][g] : 0;
    // (of the second 16 tokens: less 16, which the lanes there have in their offset)
    return (page * hk + head) * block + ((c * kChunk + u * 32) & (block - 1)) - (SMALL ? 16 * g : 0);
  };
  auto load_k = [&](int c, const Pages4& p, Raw4<DIM>& r) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const char* kp = reinterpret_cast<const char*>(a.pool.k) + tokens_before(c, p, u, 0) * (DIM / 2);
      if constexpr (SMALL) {
        const char* second = reinterpret_cast<const char*>(a.pool.k) + tokens_before(c, p, u, 1) * (DIM / 2);
        kp = rho >= 8 ? second : kp;
      }
      load_words<KW>(kp + k_at, r.k[2 * u]);
      load_words<KW>(kp + (k_at + DIM), r.k[2 * u + 1]);
    }
  };
  auto load_v = [&](int c, const Pages4& p, Raw4<DIM>& r) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int64_t at = tokens_before(c, p, u, 0);
      if constexpr (SMALL) {
        const int64_t second = tokens_before(c, p, u, 1);
        at = h >= 2 ? second : at;
      }
      const char* vp = reinterpret_cast<const char*>(a.pool.v) + at * (DIM / 2);
#pragma unroll
      for (int d = 0; d < DP; ++d) r.v[u][d] = *reinterpret_cast<const u4*>(vp + (v_at + d * 256));
      r.ks[u] = *reinterpret_cast<const u4*>(reinterpret_cast<const char*>(a.pool.k_scale + at) + static_cast<uint32_t>(16 * h));
      r.vs[u] = *reinterpret_cast<const u4*>(reinterpret_cast<const char*>(a.pool.v_scale + at) + static_cast<uint32_t>(16 * h));
    }
  };

  // the first chunk is on its way while the queries are read
  Raw4<DIM> raw;
  const int c_first = __builtin_amdgcn_readfirstlane(c_begin + wave);
  now_at = pages_of(c_first);
  Pages4 ahead = pages_of(c_first + WAVES);  // past the end: -1, or a page that is not used
  if (c_first < c_end) {
    load_k(c_first, now_at, raw);
    load_v(c_first, now_at, raw);
  }

  // query rows of this lane (one of 16 for each mt): fragments, sums, key ranges
  __shared__ u4 q_rows[MT][KW][64];  // the fragments of a wave: the same in all
  float factor[MT], start[MT];
  int from[MT], upto[MT];
  int all_from = 0, all_upto = INT_MAX;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int i = row0 + mt * 16 + rho;
    const bool real = i < sp.n * a.group;
    const int tok = real ? i / a.group : 0, hq = head * a.group + (real ? i - tok * a.group : 0);
    const uint16_t* q = a.q + static_cast<int64_t>(sp.t0 + tok) * a.q_token + static_cast<int64_t>(hq) * a.q_head;
    u4 raw[KW];
    float inverse = 1.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) raw[w] = *reinterpret_cast<const u4*>(q + h * (DIM / 4) + w * 8);
    if (a.bf16) {
      float top = 0.0f, fac;
#pragma unroll
      for (int w = 0; w < KW; ++w) top = fmaxf(top, absmax8_bf16(raw[w]));
      row_factor(max_xor16(max_xor32(top)), fac, inverse);
#pragma unroll
      for (int w = 0; w < KW; ++w) raw[w] = bf16_to_scaled_f16(raw[w], fac);
    }
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      sum += sum8_f32(raw[w]);
      if (wave == 0) q_rows[mt][w][lane] = perm_x_w4(raw[w]);
    }
    start[mt] = -add_xor16(add_xor32(sum));
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
  __syncthreads();
  all_from = __builtin_amdgcn_readfirstlane(all_from);
  all_upto = __builtin_amdgcn_readfirstlane(all_upto);

  const Fields fields;
  f4 acc[MT][4 * DP];
  float m[MT], l[MT];
  int unit[MT];  // k + 14: the exponent field of the largest scale that the row has seen
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    unit[mt] = 0;
    m[mt] = kNegInf;
    l[mt] = 0.0f;
#pragma unroll
    for (int d = 0; d < 4 * DP; ++d) acc[mt][d] = f4{0, 0, 0, 0};
  }

  // one chunk: k's registers take the next chunk's rows before the second product (not
  // before the softmax, which needs registers too: 53 and 50 us for 96 sequences of up
  // to 8192 keys), v's do after it
  auto step = [&](int c, Raw4<DIM>& r) {
    const bool more = c + WAVES < c_end;
    bool whole = (c * kChunk >= all_from) & (c * kChunk <= all_upto - kChunk);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int g = 0; g < (SMALL ? 2 : 1); ++g) whole = whole & there(c, now_at, u, g);
    f4 s[MT][4];
    h2 k_scale[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Scales8 sc = scales8(fields, r.ks[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        k_scale[u][i] = sc.scale[i];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          f4& t = s[mt][2 * u + (i >> 1)];
          t[2 * (i & 1)] = __builtin_fmaf(static_cast<float>(sc.zero64[i].x), start[mt], 0.0f);
          t[2 * (i & 1) + 1] = __builtin_fmaf(static_cast<float>(sc.zero64[i].y), start[mt], 0.0f);
        }
      }
    }
    {
      asm volatile("" ::: "memory");  // read here each time: 16 registers less
      h8 qf[MT][KW];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int w = 0; w < KW; ++w) qf[mt][w] = as_h8(q_rows[mt][w][lane]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const h8 k = fields.codes64(r.k[t][w]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qf[mt][w], s[mt][t], 0, 0, 0);
        }
    }
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        r.vs[u] = first_words(r.vs[u], lane_there(c, u) ? max(min(limit - (c * kChunk + u * 32 + 8 * h), 8), 0) : 0);
    }
    // the largest scale of the lane's tokens, as an exponent field
    const auto field_of = [](u4 x, u4 y) {
      const uint32_t big = max_pairs(max_pairs(max_pairs(x.x, x.y), max_pairs(x.z, x.w)), max_pairs(max_pairs(y.x, y.y), max_pairs(y.z, y.w)));
      return static_cast<int>(max(big & 0xFFFFu, big >> 16) >> 10);
    };
    const int all_field = field_of(r.vs[0], r.vs[1]);
    float base[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const h2 sc = k_scale[t >> 1][2 * (t & 1) + (i >> 1)];
          s[mt][t][i] *= __builtin_fmaf(static_cast<float>(i & 1 ? sc.y : sc.x), factor[mt], 0.0f);
        }
      int field = all_field;
      if (!whole) {
        u4 vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // of the lane's 8 tokens, the seen ones are `seen` from `begin` on
          const int key = c * kChunk + u * 32 + 8 * h, begin = max(from[mt] - key, 0), end = min(upto[mt] - key, 8);
          const uint32_t seen = lane_there(c, u) ? max(end - begin, 0) : 0;
          vs[u] = words_from(first_words(r.vs[u], max(end, 0)), min(begin, 8));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f4& t = s[mt][2 * u + ((j & 3) >> 1)];
            t[2 * (j & 1) + (j >> 2)] = static_cast<uint32_t>(j - begin) < seen ? t[2 * (j & 1) + (j >> 2)] : kNegInf;
          }
        }
        field = field_of(vs[0], vs[1]);
      }
      float shrink = 1.0f;
      if (__any(field > unit[mt])) {
        field = max(field, unit[mt]);
#pragma unroll
        for (int d = 16; d < 64; d *= 2) field = max(field, __shfl_xor(field, d));
        shrink = __uint_as_float(static_cast<uint32_t>(127 - (field - unit[mt])) << 23);
        unit[mt] = field;
      }
      float mx = kNegInf;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[mt][t][i]);
      float now = fmaxf(m[mt], max_xor16(max_xor32(mx)));
      // the reference moves only where weights would leave f16's range
      if (!__any(now > m[mt] + kSlack4)) now = m[mt];
      const float ref = now == kNegInf ? 0.0f : now;
      const float down = __builtin_amdgcn_exp2f(m[mt] - ref) * shrink;
      m[mt] = now;
      base[mt] = ref - (kLift + 14.0f - static_cast<float>(unit[mt]));
      if (__any(down != 1.0f)) {
        l[mt] *= down;
#pragma unroll
        for (int d = 0; d < 4 * DP; ++d) acc[mt][d] *= down;
      }
    }
    if (more) load_k(c + WAVES, ahead, r);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Scales8 sc = scales8(fields, r.vs[u]);
      u4 pf[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f4& t = s[mt][2 * u + (i >> 1)];
          const float p0 = __builtin_amdgcn_exp2f(t[2 * (i & 1)] - base[mt]), p1 = __builtin_amdgcn_exp2f(t[2 * (i & 1) + 1] - base[mt]);
          l[mt] += p0 + p1;
          const h2 pk = {static_cast<_Float16>(__builtin_fmaf(p0, static_cast<float>(sc.scale[i].x), 0.0f)),
                         static_cast<_Float16>(__builtin_fmaf(p1, static_cast<float>(sc.scale[i].y), 0.0f))};
          d[i] = as_u32(pk);
        }
        pf[mt] = u4{d[0], d[1], d[2], d[3]};
      }
#pragma unroll
      for (int d = 0; d < DP; ++d) {
        const uint32_t v[4] = {r.v[u][d].x, r.v[u][d].y, r.v[u][d].z, r.v[u][d].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const h8 codes = differences8(fields, v[e], sc);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[mt][d * 4 + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes, as_h8(pf[mt]), acc[mt][d * 4 + e], 0, 0, 0);
        }
      }
    }
    if (more) {
      load_v(c + WAVES, ahead, r);
      now_at = ahead;
      ahead = pages_of(c + 2 * WAVES);
    }
  };

  for (int c = c_first; c < c_end; c += WAVES) step(c, raw);

  // join the waves, 16 rows at a time; weights in units of 2^-kLift, whatever the scales
  const bool alone = part.splits == 1;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const float scale_unit = __uint_as_float(static_cast<uint32_t>(127 + unit[mt] - 14) << 23);
    const float weight = add_xor16(add_xor32(l[mt])) * scale_unit;
    if (h == 0) {
      join_m[wave][rho] = m[mt];
      join_l[wave][rho] = weight;
    }
    // the product's rows are values 64 d + 4 (4 h + i) + e
#pragma unroll
    for (int d = 0; d < DP; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f4*>(&join[wave][rho][d * 64 + h * 16 + i * 4]) =
            f4{acc[mt][d * 4][i], acc[mt][d * 4 + 1][i], acc[mt][d * 4 + 2][i], acc[mt][d * 4 + 3][i]} * scale_unit;
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
          y += *reinterpret_cast<const f4*>(&join[w][row][d]) * (__builtin_amdgcn_exp2f(join_m[w][row] - ref) * inv);
        if (alone) {
          const int tok = (row0 + i) / a.group, hq = head * a.group + (row0 + i) - tok * a.group;
          const int64_t at = static_cast<int64_t>(sp.t0 + tok) * a.heads + hq;
          uint16_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = a.bf16 ? f32_to_bf16_bits(y[e]) : f32_to_f16_bits(y[e]);
          *reinterpret_cast<uint2*>(a.out + at * DIM + d) =
              uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                    static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
          if (a.lse && d == 0) a.lse[at] = log_sum(ref, total);
        } else {
          const int64_t at = static_cast<int64_t>(part.base + part.nth) * kRows + i;
          *reinterpret_cast<f4*>(a.part + at * DIM + d) = y;
          if (d == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = float2{top, total};
        }
      }
    }
    if (mt + 1 < MT) __syncthreads();
  }
}

namespace {

struct Parts4 {
  // Three workgroups a compute unit are what its registers hold (three sequences of
  // 131000 keys: 90 us with three, 100 with five, 105 with eight).
  static constexpr int kPerUnit = 3, kLongChunks = INT_MAX;
  template <int DIM, int MT, int WAVES>
  static hipError_t launch(const Attend4Args& a, unsigned slots) {
    const dim3 grid(slots), block(64 * WAVES);
    if (a.pool.block == 16) hipLaunchKernelGGL((attend4_few_kernel<DIM, MT, WAVES, true>), grid, block, 0, a.stream, a);
    else hipLaunchKernelGGL((attend4_few_kernel<DIM, MT, WAVES, false>), grid, block, 0, a.stream, a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_attend4(const Attend4Args& a, const DeviceInfo& dev) { return launch_attend_parts<Parts4>(a, dev); }

}  // namespace mxq
