// Attention of many new tokens a sequence (prompts, chunks of prompts) over the
// 8-bit paged cache; the mathematics and the rounding are those of the few-row
// kernel.
//
// Bound: the matrix cores and, beside them, the exponentials (one for each
// score, against 4 * dim flops).  A workgroup holds 128 rows (query heads that
// share a kv head, times new tokens), 32 a wave, and walks the keys 64 at a
// time.  The codes of a stage become f16 once, on their way into LDS, for all
// four waves; the next stage's codes are fetched meanwhile.
//
// S^T = K Q^T on 32 x 32 tiles leaves each lane 32 of 64 scores of one query
// row: maxima and sums stay in the lane but for one exchange with lane ^ 32,
// and the probabilities are the operand of O^T = V^T P^T in place.  That operand
// holds keys 4h .. 4h+3 and 8+4h .. 8+4h+3 of 16 in half h, so v's codes are
// put into LDS in that order.  16-byte pieces are stored at piece ^ row so that
// 32 rows' reads of one column meet different banks.
//
// A weight is one fma and one exp2, v's scale being part of the exponent.  The
// reference (a row's largest score so far) moves only where a weight would
// leave f16's range, so most stages rescale nothing.  Stages on the diagonal or
// with missing pages mask their scores first; a stage with weights below f16's
// normal range (rare, or page scales far apart) adds those in products of their
// own.
//
// 32 rows a wave and 128 a workgroup: 256 rows in 8 waves stage half as often a
// row, but their barrier costs more (six chunks of prompts, 128 values a head:
// 353 against 335 us).  No vector register is spilled; 34 .. 38 scalar ones are,
// into lanes, and some are read back in the loop over stages.  Measured: a prompt
// of 4001 tokens, 32 heads of 64 values, 120 us (546 TFLOP/s; 125 .. 140 on other
// cards); six chunks of up to 1024 tokens over up to 8192 keys, 128 values, window
// 4096, 335 us (565 TFLOP/s).  On a card where they take 142 and 335: without the
// staging 113 and 255, without the exponentials 131 and 317, without the search
// for small weights 123 and 300.  The vector ALU (of which the codes' conversion
// is a fifth at 128 values) issues in 55 % (128 values) and 75 % (64) of the
// cycles, the matrix cores in 25 .. 30 %.
#include <cfloat>
#include <climits>

#include "attend_split.h"

namespace mxq {

namespace {

constexpr int kManyThreads = 256, kStage = 64;
constexpr float kTinyScale = 0x1p-100f;
constexpr float kSlack = 1.75f;  // weights reach 2^(kLift + kSlack), below f16's largest

template <int DIM>
struct Stage {
  u4 k[kStage * DIM / 8];
  u4 v[DIM * kStage / 8];
  // of the stage's 16-key groups; vs -1: no such page; with v's, its log2 and its inverse
  float ks[4], vs[4], log_vs[4], inv_vs[4];
  float pad[48];  // a stage is a multiple of 256 bytes
};

// Place of a 16-byte piece of a row.
template <int DIM>
__device__ __forceinline__ int k_at(int row, int piece) {
  return DIM == 64 ? row * 8 + (piece ^ ((row >> 1) & 7)) : row * 16 + (piece ^ (row & 15));
}
__device__ __forceinline__ int v_at(int d, int piece) { return d * 8 + (piece ^ ((d >> 1) & 7)); }

__device__ __forceinline__ float max8(const f16x& s, int from) {
  float m = fmaxf(fmaxf(s[from], s[from + 1]), s[from + 2]);
  m = fmaxf(fmaxf(m, s[from + 3]), s[from + 4]);
  m = fmaxf(fmaxf(m, s[from + 5]), s[from + 6]);
  return fmaxf(m, s[from + 7]);
}
__device__ __forceinline__ float min8(const f16x& s, int from) {
  float m = fminf(fminf(s[from], s[from + 1]), s[from + 2]);
  m = fminf(fminf(m, s[from + 3]), s[from + 4]);
  m = fminf(fminf(m, s[from + 5]), s[from + 6]);
  return fminf(m, s[from + 7]);
}

__device__ __forceinline__ u4 again(u4 w) {
  asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
  return w;
}

}  // namespace

template <int DIM, bool BF16>
__global__ __launch_bounds__(kManyThreads, 2) void attend_many_kernel(AttendArgs a) {
  constexpr int KS = DIM / 16, DB = DIM / 32, KP = DIM / 64;  // product steps, d blocks, pieces a thread stages
  extern __shared__ __align__(16) char lds[];
  Stage<DIM>* stage = reinterpret_cast<Stage<DIM>*>(lds);
  const int hk = a.pool.kv_heads, block = a.pool.block;
  // later rows see more keys: they go first
  const int unit = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  const int part = unit / hk % a.many_splits, head = unit % hk;
  int seq = 0, first = 0;
  const int tile_index = unit / hk / a.many_splits;
  if (!find_tile(a, tile_index, seq, first)) return;
  seq = __builtin_amdgcn_readfirstlane(seq);
  first = __builtin_amdgcn_readfirstlane(first);
  SeqSpan sp = seq_span(a, seq);
  sp.t0 = __builtin_amdgcn_readfirstlane(sp.t0);
  sp.n = __builtin_amdgcn_readfirstlane(sp.n);
  sp.len = __builtin_amdgcn_readfirstlane(sp.len);
  const int row0 = (tile_index - first) * kManyRows, rows = sp.n * a.group;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 31, h = lane >> 5;
  const int limit = min(sp.len, a.width * block), pos0 = sp.len - sp.n;

  // this lane's query row; rows past the last repeat it and are not stored
  const int mine = row0 + wave * 32 + col, row = min(mine, rows - 1);
  const int tok = row / a.group, hq = head * a.group + row - tok * a.group;
  const int pos = pos0 + tok;
  const int upto = min(pos + 1, limit), from = first_seen(a, pos);
  u4 qf[KS];
  {
    const uint16_t* q = a.q + static_cast<int64_t>(sp.t0 + tok) * a.q_token + static_cast<int64_t>(hq) * a.q_head;
#pragma unroll
    for (int i = 0; i < KS; ++i) qf[i] = *reinterpret_cast<const u4*>(q + i * 16 + h * 8);
  }
  float inverse = 1.0f;
  if constexpr (BF16) {
    float top = 0.0f, fac;
#pragma unroll
    for (int i = 0; i < KS; ++i) top = fmaxf(top, absmax8_bf16(qf[i]));
    row_factor(max_xor32(top), fac, inverse);
#pragma unroll
    for (int i = 0; i < KS; ++i) qf[i] = bf16_to_scaled_f16(qf[i], fac);
  }
  // the softmax's scale is taken positive: largest scores are looked for before it is applied
  if (a.scale2 < 0.0f) {
#pragma unroll
    for (int i = 0; i < KS; ++i) qf[i] ^= 0x80008000u;
  }
  const float factor = fabsf(a.scale2) * inverse;

  // the wave's rows are in order: its first and last hold the narrowest and widest ranges
  const int last_row = min(row0 + wave * 32 + 31, rows - 1), first_row = min(row0 + wave * 32, rows - 1);
  const int pos_lo = pos0 + first_row / a.group, pos_hi = pos0 + last_row / a.group;
  // a wave without rows takes no part but in the staging
  const int wave_upto = row0 + wave * 32 < rows ? min(pos_hi + 1, limit) : 0, wave_from = first_seen(a, pos_lo);
  const int all_upto = min(pos_lo + 1, limit), all_from = first_seen(a, pos_hi);

  // the tile's stages, and this part's share of them
  const int tile_last = min(row0 + kManyRows, rows) - 1;
  const int key_hi = min(pos0 + tile_last / a.group + 1, limit);
  const int key_lo = first_seen(a, pos0 + row0 / a.group);
  const int s_lo = key_lo / kStage, s_hi = max(s_lo, key_hi / kStage + (key_hi % kStage > 0));
  const int per = (s_hi - s_lo + a.many_splits - 1) / a.many_splits;
  const int begin = min(s_lo + part * per, s_hi), end = min(begin + per, s_hi);

  // staging: K rows of 16 codes, V rows of 16 tokens
  const int32_t* table = a.table + static_cast<int64_t>(seq) * a.table_stride;
  constexpr int kPer = DIM / 16;           // pieces of a K row
  const int kr = tid / kPer, kc = tid % kPer, vd = tid >> 2, vg = tid & 3;
  u4 kraw[KP], vraw[KP];
  float ks = 0.0f, vs = 0.0f;
  int pk[KP], pv;
  const int block_log2 = 31 - __builtin_clz(block);
  const uint32_t page_bytes = static_cast<uint32_t>(hk) * block * DIM;  // hk < 2^16, a page of a head at most 2^14
  const int8_t* k_base = a.pool.k + static_cast<int64_t>(head) * block * DIM + kc * 16;
  const int8_t* v_base = a.pool.v + (static_cast<int64_t>(head) * DIM + vd) * block;
  const uint32_t nb = static_cast<uint32_t>(a.pool.blocks);
  auto pages = [&](int s) {
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const int at = (s * kStage + kr + j * (256 / kPer)) >> block_log2;
      pk[j] = at < a.width ? table[at] : -1;
    }
    const int at = (s * kStage + vg * 16) >> block_log2;
    pv = at < a.width ? table[at] : -1;
  };
  auto fetch = [&](int s) {
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const uint32_t p = static_cast<uint32_t>(pk[j]) < nb ? pk[j] : 0;
      const int t = (s * kStage + kr + j * (256 / kPer)) & (block - 1);
      kraw[j] = *reinterpret_cast<const u4*>(k_base + static_cast<uint64_t>(p) * page_bytes + static_cast<uint32_t>(t * DIM));
    }
    // a page past the sequence's end may be anyone's, or never written
    const bool ok = static_cast<uint32_t>(pv) < nb && s * kStage + vg * 16 < limit;
    const uint32_t p = ok ? pv : 0;
    const int8_t* vp = v_base + static_cast<uint64_t>(p) * page_bytes + ((s * kStage + vg * 16) & (block - 1));
#pragma unroll
    for (int j = 0; j < KP; ++j) vraw[j] = *reinterpret_cast<const u4*>(vp + j * 64 * block);
    if (tid < 4) {
      ks = ok ? a.pool.k_scale[static_cast<int64_t>(p) * hk + head] : 0.0f;
      vs = ok ? a.pool.v_scale[static_cast<int64_t>(p) * hk + head] : -1.0f;
    }
  };
  const uint32_t magic = kMagic;
  auto put = [&](Stage<DIM>& st) {
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const int r = kr + j * (256 / kPer), d = vd + j * 64;
      st.k[k_at<DIM>(r, 2 * kc)] = codes8_f16(kraw[j].x, kraw[j].y, magic);
      st.k[k_at<DIM>(r, 2 * kc + 1)] = codes8_f16(kraw[j].z, kraw[j].w, magic);
      st.v[v_at(d, 2 * vg)] = codes8_f16(vraw[j].x, vraw[j].z, magic);
      st.v[v_at(d, 2 * vg + 1)] = codes8_f16(vraw[j].y, vraw[j].w, magic);
    }
    if (tid < 4) {
      st.ks[tid] = ks;
      st.vs[tid] = vs;
      // what a page without a scale (or a tiny one) holds is masked, or takes the rare way
      st.log_vs[tid] = vs < 0.0f ? 0.0f : __builtin_amdgcn_logf(vs);  // log2
      st.inv_vs[tid] = vs >= FLT_MIN ? __builtin_amdgcn_rcpf(vs) : 0.0f;
    }
  };

  f16x acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[db][i] = 0.0f;
  float m = kNegInf, l = 0.0f, top_vs = kTinyScale, log_top_vs = -100.0f;

  // LDS addresses of this lane's operands: piece ^ row, so a step along the row
  // is an xor of the whole address (rows are 128 or 256 bytes, stages multiples of them)
  const uint32_t k_first = static_cast<uint32_t>(k_at<DIM>(col, h)) * 16, v_first = static_cast<uint32_t>(v_at(col, h)) * 16 + kStage * DIM * 2;
  auto compute = [&](int s, int at) {
    const Stage<DIM>& st = stage[at];
    const uint32_t k_row = k_first + static_cast<uint32_t>(at) * sizeof(Stage<DIM>), v_row = v_first + static_cast<uint32_t>(at) * sizeof(Stage<DIM>);
    auto k_piece = [&](int b, int i) { return *reinterpret_cast<const u4*>(lds + (k_row ^ (i * 32u)) + b * 64 * DIM); };
    auto v_piece = [&](int db, int g) { return *reinterpret_cast<const u4*>(lds + (v_row ^ (g * 32u)) + db * 32 * kStage * 2); };
    f16x x[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[b][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
        x[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(k_piece(b, i)), as_h8(qf[i]), x[b], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    float c[4], v[4], mx = kNegInf, shrink = 1.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      c[g] = st.ks[g] * factor;
      v[g] = st.vs[g];
    }
    const float largest = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
    const bool grows = __any(largest > top_vs);  // the same in the whole workgroup
    if (grows) {
      shrink = top_vs / largest;
      top_vs = largest;
      log_top_vs = __builtin_amdgcn_logf(largest);
    }
    const bool there = __all(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])) >= 0.0f);
    const bool masked = !(there && s * kStage >= all_from && s * kStage <= all_upto - kStage);
    if (masked) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int g = 2 * b + (i >> 3), key = s * kStage + b * 32 + 8 * (i >> 2) + 4 * h + (i & 3);
          const bool seen = v[g] >= 0.0f && key >= from && key < upto;
          x[b][i] = seen ? x[b][i] * c[g] : kNegInf;
        }
#pragma unroll
      for (int g = 0; g < 4; ++g) c[g] = 1.0f;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) mx = fmaxf(mx, max8(x[g >> 1], (g & 1) * 8) * c[g]);
    float now = fmaxf(m, max_xor32(mx));
    // the reference moves only where weights would leave f16's range: not at all for most stages
    if (!__any(now > m + kSlack)) now = m;
    const float ref = now == kNegInf ? 0.0f : now, lift = kLift - ref;
    const float alpha = __builtin_amdgcn_exp2f(m - ref), down = alpha * shrink;
    m = now;
    float off[4], mn = -kNegInf;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      off[g] = st.log_vs[g] + (lift - log_top_vs);
      if (masked) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = x[g >> 1][(g & 1) * 8 + i];
          mn = fminf(mn, e == kNegInf ? -kNegInf : e + off[g]);
        }
      } else {
        mn = fminf(mn, __builtin_fmaf(min8(x[g >> 1], (g & 1) * 8), c[g], off[g]));
      }
    }
    const bool rare = !__all(mn >= -14.0f);
    if (__any(down != 1.0f)) {
      l *= alpha;
#pragma unroll
      for (int db = 0; db < DB; ++db) acc[db] *= down;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      // (finite: a group that is masked throughout has the sum 0, whatever its page's scale is)
      float p[8], sum = 0.0f, weigh = fminf(top_vs * st.inv_vs[g], FLT_MAX);
      if (rare) {
        off[g] = lift;
        weigh = 1.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[g >> 1][8 * (g & 1) + i], c[g], off[g]));
        p[i + 1] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[g >> 1][8 * (g & 1) + i + 1], c[g], off[g]));
        sum += p[i] + p[i + 1];
      }
      l = __builtin_fmaf(sum, weigh, l);
      asm volatile("" : "+v"(l));  // added here, not where 32 weights would have to be kept for it
      if (rare) {
        const float share = fmaxf(v[g], 0.0f) / top_vs;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] *= share;
          x[g >> 1][8 * (g & 1) + i] = p[i];
          p[i] = p[i] < kF16Normal ? 0.0f : p[i];  // a NaN stays
        }
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const h2 pk2 = {static_cast<_Float16>(p[i]), static_cast<_Float16>(p[i + 1])};
        w[i / 2] = as_u32(pk2);
      }
      const h8 pf = as_h8(u4{w[0], w[1], w[2], w[3]});
#pragma unroll
      for (int db = 0; db < DB; ++db)
        acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(v_piece(db, g)), pf, acc[db], 0, 0, 0);
    }
    if (!rare) return;
    // the weights of [2^-38, 2^-14), then those 2^24 times smaller, .., until none is left
    Band band;
#pragma clang loop unroll(disable)
    for (bool more = true; more; band.next()) {
      bool left = false;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float p0 = x[g >> 1][(g & 1) * 8 + i], p1 = x[g >> 1][(g & 1) * 8 + i + 1];
          left |= band.below(p0) || band.below(p1);
          const h2 pk2 = {static_cast<_Float16>(band.lifted(p0)), static_cast<_Float16>(band.lifted(p1))};
          w[i / 2] = as_u32(pk2);
        }
        const h8 pf = as_h8(u4{w[0], w[1], w[2], w[3]});
#pragma unroll
        for (int db = 0; db < DB; ++db) {
          f16x t;
#pragma unroll
          for (int i = 0; i < 16; ++i) t[i] = 0.0f;
          t = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(again(v_piece(db, g))), pf, t, 0, 0, 0);
          acc[db] += t * (1.0f / band.lift);
          __builtin_amdgcn_sched_barrier(0);  // one product's registers at a time
        }
      }
      more = __any(left && !band.last());
    }
  };

  if (begin < end) {
    pages(begin);
    fetch(begin);
    put(stage[0]);
    pages(min(begin + 1, end - 1));
    __syncthreads();
    for (int s = begin; s < end; ++s) {
      const int at = (s - begin) & 1;
      const bool next = s + 1 < end;
      if (next) {
        fetch(s + 1);
        pages(min(s + 2, end - 1));
      }
      if (s * kStage < wave_upto && s * kStage > wave_from - kStage) compute(s, at);
      if (next) put(stage[at ^ 1]);
      __syncthreads();
    }
  }

  const float total = add_xor32(l), inv = over(total);
  if (mine >= rows) return;
  if (a.many_splits == 1) {
    const int64_t at = static_cast<int64_t>(sp.t0 + tok) * a.heads + hq;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(acc[db][4 * i + e] * inv * top_vs);
        *reinterpret_cast<uint2*>(a.out + at * DIM + db * 32 + 8 * i + 4 * h) =
            uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                  static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
      }
    if (a.lse && h == 0) a.lse[at] = log_sum(m == kNegInf ? 0.0f : m, total);
  } else {
    const int64_t at = static_cast<int64_t>(unit) * kManyRows + wave * 32 + col;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f4*>(a.many_part + at * DIM + db * 32 + 8 * i + 4 * h) =
            f4{acc[db][4 * i], acc[db][4 * i + 1], acc[db][4 * i + 2], acc[db][4 * i + 3]} * inv * top_vs;
    if (h == 0) *reinterpret_cast<float2*>(a.many_ml + at * 2) = float2{m, total};
  }
}

namespace {

template <int DIM, bool BF16>
hipError_t launch_many_of(const AttendArgs& a, unsigned grid) {
  const auto kernel = attend_many_kernel<DIM, BF16>;
  const size_t lds = 2 * sizeof(Stage<DIM>);
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kManyThreads), lds, a.stream, a);
  hipError_t le = hipGetLastError();
  if (le != hipSuccess || a.many_splits == 1) return le;
  constexpr int kHeads = 256 / (DIM / 4);
  hipLaunchKernelGGL((attend_many_join_kernel<DIM, BF16, AttendArgs>), dim3(static_cast<unsigned>(a.tokens), static_cast<unsigned>((a.heads + kHeads - 1) / kHeads)),
                     dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_many(const AttendArgs& given, float* ws) {
  AttendArgs a = given;
  const int64_t grid = many_tiles(a) * a.pool.kv_heads * a.many_splits;
  if (grid == 0) return hipSuccess;
  a.many_part = ws;
  a.many_units = static_cast<int>(grid);
  a.many_ml = ws + grid * kManyRows * a.pool.dim;
  const unsigned g = static_cast<unsigned>(grid);
  if (a.pool.dim == 64) return a.bf16 ? launch_many_of<64, true>(a, g) : launch_many_of<64, false>(a, g);
  return a.bf16 ? launch_many_of<128, true>(a, g) : launch_many_of<128, false>(a, g);
}

}  // namespace mxq
