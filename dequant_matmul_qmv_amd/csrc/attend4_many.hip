// Attention of many new tokens a sequence (prompts, chunks of prompts) over the
// 4-bit paged cache; the mathematics is that of the few-row kernel.
//
// Bound: the matrix cores and, beside them, the exponentials (one for each score,
// against 4 * dim flops): a prompt of 4001 tokens of 32 heads of 64 takes 112 .. 116 us
// (49 at a library product's rate), six chunks of heads of 128 304 .. 310 (135).  A workgroup holds 128 rows (query heads that share a kv
// head, times new tokens), 32 a wave, and walks the keys 64 at a time.  A stage's
// codes become their values, exact in f16, on their way into LDS for all four waves;
// the next stage's words are fetched meanwhile.
//
// S^T = K Q^T on 32 x 32 tiles leaves each lane 32 of 64 scores of one query row:
// maxima and sums stay in the lane but for one exchange with lane ^ 32.  Keys go to
// the rows of LDS at which a lane's 8 scores of 16 keys are the 8 tokens of a word of
// v, in the order in which its codes unpack: the weights are then the operand of
// O^T = V^T P^T in place.  q's values are taken in the order in which k's unpack.
// 16-byte pieces are stored at piece ^ row so that reads and writes of a column meet
// different banks.
//
// A weight is one fma and one exp2.  The reference (a row's largest score so far)
// moves only where a weight would leave f16's range, so most stages rescale nothing.
// Stages on the diagonal or with missing pages mask their scores first.
#include <climits>

#include "attend4_device.h"

namespace mxq {

namespace {

constexpr int kManyThreads = 256, kStage = 64;
constexpr float kSlack = 1.75f;  // weights reach 2^(kLift + kSlack), below f16's largest

template <int DIM>
struct Stage4 {
  u4 k[kStage * DIM / 8];
  u4 v[DIM * kStage / 8];
  int there[4];  // of the stage's 16-key groups: their page is
  int pad[60];   // a stage is a multiple of 256 bytes
};

// Place of a 16-byte piece of a row.
template <int DIM>
__device__ __forceinline__ int k_at(int row, int piece) {
  return DIM == 64 ? row * 8 + (piece ^ ((row >> 1) & 7)) : row * 16 + (piece ^ (row & 15));
}
__device__ __forceinline__ int v_at(int d, int piece) { return d * 8 + (piece ^ ((d >> 1) & 7) ^ ((d >> 4) & 1)); }

__device__ __forceinline__ float max8(const f16x& s, int from) {
  float m = fmaxf(fmaxf(s[from], s[from + 1]), s[from + 2]);
  m = fmaxf(fmaxf(m, s[from + 3]), s[from + 4]);
  m = fmaxf(fmaxf(m, s[from + 5]), s[from + 6]);
  return fmaxf(m, s[from + 7]);
}

}  // namespace

template <int DIM, bool BF16>
__global__ __launch_bounds__(kManyThreads, 2) void attend4_many_kernel(Attend4Args a) {
  constexpr int KS = DIM / 16, DB = DIM / 32, W = DIM / 32;  // product steps, d blocks, words of k and of v a thread stages
  extern __shared__ __align__(16) char lds[];
  Stage4<DIM>* stage = reinterpret_cast<Stage4<DIM>*>(lds);
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
  const uint32_t sign = a.scale2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
  for (int i = 0; i < KS; ++i) qf[i] = perm_x_w4(qf[i] ^ sign);
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

  // staging: a thread has W words of a key, and W words of 8 tokens
  const int32_t* table = a.table + static_cast<int64_t>(seq) * a.table_stride;
  const int kt = tid >> 2, kc = tid & 3, vg = tid >> 5, vd = (tid & 31) * W;
  // the row of S^T at which key kt's score is where its token is in a word of v
  const int place = 2 * (kt & 3) + ((kt >> 2) & 1), kr = (kt & ~15) + 4 * ((kt >> 3) & 1) + (place & 3) + 8 * (place >> 2);
  uint32_t kraw[W], vraw[W];
  uint16_t ks = 0;
  u4 vs = u4{0, 0, 0, 0};
  int pk = -1, pv = -1, valid = 0;  // the next stage's pages; of a group's 8 tokens, those that are there
  const int block_log2 = 31 - __builtin_clz(block);
  const uint32_t nb = static_cast<uint32_t>(a.pool.blocks);
  auto pages = [&](int s) {
    int at = (s * kStage + kt) >> block_log2;
    pk = at < a.width ? table[at] : -1;
    at = (s * kStage + vg * 8) >> block_log2;
    pv = at < a.width ? table[at] : -1;
  };
  auto load_words = [&](const uint32_t* p, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
      const u4 x = *reinterpret_cast<const u4*>(p);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    }
  };
  // what is fetched is first looked at by `put`, after the products of the stage before
  auto fetch = [&](int s) {
    // a page past the sequence's end may be anyone's, or never written
    const int key = s * kStage + vg * 8;
    const bool ok = static_cast<uint32_t>(pv) < nb && key < limit;
    const int64_t p = static_cast<uint32_t>(pk) < nb ? pk : 0, q = ok ? pv : 0;
    const int64_t k_token = (p * hk + head) << block_log2, v_token = (q * hk + head) << block_log2;
    const uint32_t k_slot = (s * kStage + kt) & (block - 1), v_slot = key & (block - 1);
    load_words(a.pool.k + k_token * (DIM / 8) + (k_slot * (DIM / 8) + kc * W), kraw);
    ks = (a.pool.k_scale + k_token)[k_slot];
    load_words(a.pool.v + v_token * (DIM / 8) + (v_slot * (DIM / 8) + vd), vraw);
    vs = *reinterpret_cast<const u4*>(a.pool.v_scale + v_token + v_slot);
    valid = ok ? max(min(limit - key, 8), 0) : 0;
  };
  const Fields fields;
  auto put = [&](Stage4<DIM>& st) {
    if (__any(valid < 8)) vs = first_words(vs, valid);
    const uint32_t both = ks * 0x10001u;
    const h2 scale = as_h2(both & 0x7FF07FF0u), zero = fields.with64(both << 4);
    const Scales8 k_scales{{scale, scale, scale, scale}, {zero, zero, zero, zero}}, v_scales = scales8(fields, vs);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      st.k[k_at<DIM>(kr, kc * W + w)] = __builtin_bit_cast(u4, values8(fields, kraw[w], k_scales));
      st.v[v_at(vd + w, vg)] = __builtin_bit_cast(u4, values8(fields, vraw[w], v_scales));
    }
    if ((tid & 63) == 0) st.there[tid >> 6] = valid > 0;  // of both 8-token groups: a page has 16 tokens at least
  };

  f16x acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[db][i] = 0.0f;
  float m = kNegInf, l = 0.0f;

  // LDS addresses of this lane's operands: piece ^ row, so a step along the row
  // is an xor of the whole address (rows are 128 or 256 bytes, stages multiples of them)
  const uint32_t k_first = static_cast<uint32_t>(k_at<DIM>(col, h)) * 16, v_first = static_cast<uint32_t>(v_at(col, h)) * 16 + kStage * DIM * 2;
  auto compute = [&](int s, int at) {
    const Stage4<DIM>& st = stage[at];
    const uint32_t k_row = k_first + static_cast<uint32_t>(at) * sizeof(Stage4<DIM>), v_row = v_first + static_cast<uint32_t>(at) * sizeof(Stage4<DIM>);
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
    const bool all_there = st.there[0] && st.there[1] && st.there[2] && st.there[3];
    float c = factor, mx = kNegInf;
    if (!(all_there && s * kStage >= all_from && s * kStage <= all_upto - kStage)) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        // of the lane's 8 tokens, the seen ones are `seen` from `begin` on
        const int key = s * kStage + g * 16 + 8 * h, begin = max(from - key, 0), end = min(upto - key, 8);
        const uint32_t seen = st.there[g] ? max(end - begin, 0) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * (g & 1) + j, token = (j >> 1) + 4 * (j & 1);
          x[g >> 1][i] = static_cast<uint32_t>(token - begin) < seen ? x[g >> 1][i] * factor : kNegInf;
        }
      }
      c = 1.0f;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) mx = fmaxf(mx, max8(x[g >> 1], (g & 1) * 8));
    float now = fmaxf(m, max_xor32(mx) * c);
    // the reference moves only where weights would leave f16's range: not at all for most stages
    if (!__any(now > m + kSlack)) now = m;
    const float ref = now == kNegInf ? 0.0f : now, lift = kLift - ref;
    const float alpha = __builtin_amdgcn_exp2f(m - ref);
    m = now;
    if (__any(alpha != 1.0f)) {
      l *= alpha;
#pragma unroll
      for (int db = 0; db < DB; ++db) acc[db] *= alpha;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float p[8], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[g >> 1][8 * (g & 1) + i], c, lift));
        p[i + 1] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[g >> 1][8 * (g & 1) + i + 1], c, lift));
        sum += p[i] + p[i + 1];
      }
      l += sum;
      asm volatile("" : "+v"(l));  // added here, not where 32 weights would have to be kept for it
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
        for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(acc[db][4 * i + e] * inv);
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
            f4{acc[db][4 * i], acc[db][4 * i + 1], acc[db][4 * i + 2], acc[db][4 * i + 3]} * inv;
    if (h == 0) *reinterpret_cast<float2*>(a.many_ml + at * 2) = float2{m, total};
  }
}

namespace {

template <int DIM, bool BF16>
hipError_t launch_many_of(const Attend4Args& a, unsigned grid) {
  const auto kernel = attend4_many_kernel<DIM, BF16>;
  const size_t lds = 2 * sizeof(Stage4<DIM>);
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kManyThreads), lds, a.stream, a);
  hipError_t le = hipGetLastError();
  if (le != hipSuccess || a.many_splits == 1) return le;
  constexpr int kHeads = 256 / (DIM / 4);
  hipLaunchKernelGGL((attend_many_join_kernel<DIM, BF16, Attend4Args>), dim3(static_cast<unsigned>(a.tokens), static_cast<unsigned>((a.heads + kHeads - 1) / kHeads)),
                     dim3(256), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_many(const Attend4Args& given, float* ws) {
  Attend4Args a = given;
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
