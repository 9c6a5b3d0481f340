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
// A stage that every row of the wave sees, with nothing unusual, takes the short
// way: p * vscale share is one fma and one exp2, the share being part of the
// exponent.  Others (the diagonal, missing pages, weights below f16's normal
// range, page scales far apart) take each score apart.
#include <climits>

#include "attend_device.h"

namespace mxq {

namespace {

constexpr int kManyThreads = 256, kManyRows = 128, kStage = 64;
constexpr float kTinyScale = 1e-30f;

template <int DIM>
struct Stage {
  u4 k[kStage * DIM / 8];
  u4 v[DIM * kStage / 8];
  float ks[4], vs[4];  // of the stage's 16-key groups; vs -1: no such page
  float pad[56];       // a stage is a multiple of 256 bytes
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

// Rows a sequence gives to this kernel, in tiles.
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int s) {
  if (s >= a.seqs) return 0;
  const SeqSpan q = seq_span(a, s);
  const int64_t rows = static_cast<int64_t>(q.n) * a.group;
  return rows > a.few_rows ? static_cast<int>((rows + kManyRows - 1) / kManyRows) : 0;
}

}  // namespace

// (sequence, tile within it) of tile `index`, or with index < 0 the first tile
// of sequence `seq` in `first`.  Whole waves.
__device__ bool find_tile(const AttendArgs& a, int index, int& seq, int& first) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const int count = tiles_of(a, s0 + lane);
    int sum = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const unsigned long long hit = index >= 0 ? __ballot(before + sum > index) : (seq < s0 + 64 ? 1ull << (seq - s0) : 0);
    if (hit != 0) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      seq = s0 + src;
      first = before + __shfl(sum, src) - __shfl(count, src);
      return true;
    }
    before += __shfl(sum, 63);
  }
  return false;
}

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
  const SeqSpan sp = seq_span(a, seq);
  const int row0 = (tile_index - first) * kManyRows, rows = sp.n * a.group;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 31, h = lane >> 5;
  const int limit = min(max(sp.len, 0), a.width * block), pos0 = sp.len - sp.n;

  // this lane's query row; rows past the last repeat it and are not stored
  const int mine = row0 + wave * 32 + col, row = min(mine, rows - 1);
  const int tok = row / a.group, hq = head * a.group + row - tok * a.group;
  const int pos = pos0 + tok;
  const int upto = min(pos + 1, limit), from = a.window > 0 ? max(0, pos - a.window + 1) : 0;
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
  const int wave_upto = min(pos_hi + 1, limit), wave_from = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;
  const int all_upto = min(pos_lo + 1, limit), all_from = a.window > 0 ? max(0, pos_hi - a.window + 1) : 0;

  // the tile's stages, and this part's share of them
  const int tile_last = min(row0 + kManyRows, rows) - 1;
  const int key_hi = min(pos0 + tile_last / a.group + 1, limit);
  const int key_lo = a.window > 0 ? max(0, pos0 + row0 / a.group - a.window + 1) : 0;
  const int s_lo = key_lo / kStage, s_hi = max(s_lo, (key_hi + kStage - 1) / kStage);
  const int per = (s_hi - s_lo + a.many_splits - 1) / a.many_splits;
  const int begin = min(s_lo + part * per, s_hi), end = min(begin + per, s_hi);

  // staging: K rows of 16 codes, V rows of 16 tokens
  const int32_t* table = a.table + static_cast<int64_t>(seq) * a.table_stride;
  constexpr int kPer = DIM / 16;           // pieces of a K row
  const int kr = tid / kPer, kc = tid % kPer, vd = tid >> 2, vg = tid & 3;
  u4 kraw[KP], vraw[KP];
  float ks = 0.0f, vs = 0.0f;
  int pk[KP], pv;
  auto pages = [&](int s) {
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const int at = (s * kStage + kr + j * (256 / kPer)) / block;
      pk[j] = at < a.width ? table[at] : -1;
    }
    const int at = (s * kStage + vg * 16) / block;
    pv = at < a.width ? table[at] : -1;
  };
  auto fetch = [&](int s) {
    const int nb = static_cast<int>(a.pool.blocks);
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const int64_t p = pk[j] >= 0 && pk[j] < nb ? pk[j] : 0;
      const int t = (s * kStage + kr + j * (256 / kPer)) & (block - 1);
      kraw[j] = *reinterpret_cast<const u4*>(a.pool.k + ((p * hk + head) * block + t) * DIM + kc * 16);
    }
    // a page past the sequence's end may be anyone's, or never written
    const bool ok = pv >= 0 && pv < nb && s * kStage + vg * 16 < limit;
    const int64_t p = ok ? pv : 0;
    const int t = (s * kStage + vg * 16) & (block - 1);
#pragma unroll
    for (int j = 0; j < KP; ++j)
      vraw[j] = *reinterpret_cast<const u4*>(a.pool.v + ((p * hk + head) * DIM + vd + j * 64) * block + t);
    if (tid < 4) {
      ks = ok ? a.pool.k_scale[p * hk + head] : 0.0f;
      vs = ok ? a.pool.v_scale[p * hk + head] : -1.0f;
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
    }
  };

  f16x acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[db][i] = 0.0f;
  float m = kNegInf, l = 0.0f, top_vs = kTinyScale;

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
    float c[4], v[4], mx = kNegInf;
    bool ok = true;
    const float was_vs = top_vs;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      c[g] = st.ks[g] * factor;
      v[g] = st.vs[g];
      ok = ok && v[g] >= 0.0f;
      top_vs = fmaxf(top_vs, v[g]);
    }
    const float inv_vs = 1.0f / top_vs, shrink = was_vs * inv_vs;
    bool plain = ok && s * kStage >= all_from && (s + 1) * kStage <= all_upto;
    float off[4], sh[4];
    if (plain) {
      float mn = -kNegInf;
#pragma unroll
      for (int g = 0; g < 4; ++g) mx = fmaxf(mx, max8(x[g >> 1], (g & 1) * 8) * c[g]);
      const float now = fmaxf(m, max_xor32(mx));
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        sh[g] = v[g] * inv_vs;
        off[g] = __builtin_amdgcn_logf(sh[g]) + (kLift - now);  // log2
        mn = fminf(mn, __builtin_fmaf(min8(x[g >> 1], (g & 1) * 8), c[g], off[g]));
      }
      plain = __all(mn >= -14.0f && now > kNegInf);  // and no NaN
      if (plain) {
        const float alpha = __builtin_amdgcn_exp2f(m - now), down = alpha * shrink;
        m = now;
        l *= alpha;
        if (__any(down != 1.0f)) {
#pragma unroll
          for (int db = 0; db < DB; ++db) acc[db] *= down;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int g = 2 * b + j;
            float sum = 0.0f;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b][8 * j + i], c[g], off[g]));
              const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b][8 * j + i + 1], c[g], off[g]));
              sum += p0 + p1;
              const h2 pk2 = {static_cast<_Float16>(p0), static_cast<_Float16>(p1)};
              w[i / 2] = as_u32(pk2);
            }
            l = __builtin_fmaf(sum, 1.0f / sh[g], l);
            const h8 pf = as_h8(u4{w[0], w[1], w[2], w[3]});
#pragma unroll
            for (int db = 0; db < DB; ++db)
              acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(v_piece(db, g)), pf, acc[db], 0, 0, 0);
          }
        return;
      }
    }
    // each score apart
    mx = kNegInf;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int g = 2 * b + (i >> 3), key = s * kStage + b * 32 + 8 * (i >> 2) + 4 * h + (i & 3);
        const bool seen = v[g] >= 0.0f && key >= from && key < upto;
        x[b][i] = seen ? x[b][i] * c[g] : kNegInf;
        mx = fmaxf(mx, x[b][i]);
      }
    const float now = fmaxf(m, max_xor32(mx)), ref = now == kNegInf ? 0.0f : now;
    const float alpha = __builtin_amdgcn_exp2f(m - ref), down = alpha * shrink;
    m = now;
    l *= alpha;
#pragma unroll
    for (int db = 0; db < DB; ++db) acc[db] *= down;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float share = fmaxf(v[g], 0.0f) * inv_vs;
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(x[g >> 1][(g & 1) * 8 + i] - ref + kLift);
        l += p[i];
        p[i] *= share;
      }
      // the weights of [2^-14, ..), then those 2^24, 2^48, .. times smaller, until none is left
      float ceiling = -kNegInf, floor = kF16Normal, lift = 1.0f;
      for (bool more = true; more; ceiling = floor, floor *= 1.0f / kLowLift, lift *= kLowLift) {
        bool left = false;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          left = left || (p[i] > 0.0f && p[i] < floor) || (p[i + 1] > 0.0f && p[i + 1] < floor);
          // a NaN belongs to the first round
          const bool in0 = lift == 1.0f ? !(p[i] < floor) : p[i] < ceiling && p[i] >= floor;
          const bool in1 = lift == 1.0f ? !(p[i + 1] < floor) : p[i + 1] < ceiling && p[i + 1] >= floor;
          const h2 pk2 = {static_cast<_Float16>(in0 ? p[i] * lift : 0.0f), static_cast<_Float16>(in1 ? p[i + 1] * lift : 0.0f)};
          w[i / 2] = as_u32(pk2);
        }
        const h8 pf = as_h8(u4{w[0], w[1], w[2], w[3]});
        more = __any(left);
#pragma unroll
        for (int db = 0; db < DB; ++db) {
          f16x t;
#pragma unroll
          for (int i = 0; i < 16; ++i) t[i] = 0.0f;
          t = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(again(v_piece(db, g))), pf, t, 0, 0, 0);
          acc[db] += t * (1.0f / lift);
          __builtin_amdgcn_sched_barrier(0);  // one product's registers at a time
        }
      }
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
      if (s * kStage < wave_upto && (s + 1) * kStage > wave_from) compute(s, at);
      if (next) put(stage[at ^ 1]);
      __syncthreads();
    }
  }

  const float total = add_xor32(l);
  if (mine >= rows) return;
  if (a.many_splits == 1) {
    const int64_t at = static_cast<int64_t>(sp.t0 + tok) * a.heads + hq;
    const float inv = total > 0.0f || total != total ? top_vs / total : 0.0f;
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
            f4{acc[db][4 * i], acc[db][4 * i + 1], acc[db][4 * i + 2], acc[db][4 * i + 3]} * top_vs;
    if (h == 0) *reinterpret_cast<float2*>(a.many_ml + at * 2) = float2{m, total};
  }
}

// Joins a row's parts where the key axis was split: one workgroup of DIM / 4
// lanes for each (token, query head).
template <int DIM, bool BF16>
__global__ __launch_bounds__(64) void attend_many_join_kernel(AttendArgs a) {
  const int tok = blockIdx.x, hq = blockIdx.y, hk = a.pool.kv_heads, head = hq / a.group;
  int lo = 0, hi = a.seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.starts[mid] <= tok) lo = mid; else hi = mid;
  }
  int seq = lo, first = 0;
  const SeqSpan sp = seq_span(a, seq);
  if (tok < sp.t0 || tok >= sp.t0 + sp.n || static_cast<int64_t>(sp.n) * a.group <= a.few_rows) return;
  find_tile(a, -1, seq, first);
  const int i = (tok - sp.t0) * a.group + hq - head * a.group;
  const int64_t tile = first + i / kManyRows;
  const int d = threadIdx.x * 4;
  if (d >= DIM) return;
  float top = kNegInf, total = 0.0f;
  f4 y = f4{0, 0, 0, 0};
  for (int s = 0; s < a.many_splits; ++s) {
    const int64_t at = ((tile * a.many_splits + s) * hk + head) * kManyRows + i % kManyRows;
    const float2 ml = *reinterpret_cast<const float2*>(a.many_ml + at * 2);
    const f4 v = *reinterpret_cast<const f4*>(a.many_part + at * DIM + d);
    const float now = fmaxf(top, ml.x), ref = now == kNegInf ? 0.0f : now;
    const float e0 = __builtin_amdgcn_exp2f(top - ref), e1 = __builtin_amdgcn_exp2f(ml.x - ref);
    y = y * e0 + v * e1;
    total = total * e0 + ml.y * e1;
    top = now;
  }
  const int64_t at = static_cast<int64_t>(tok) * a.heads + hq;
  const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
  uint16_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(y[e] * inv);
  *reinterpret_cast<uint2*>(a.out + at * DIM + d) = uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                                                          static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
  if (a.lse && d == 0) a.lse[at] = log_sum(top == kNegInf ? 0.0f : top, total);
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
  hipLaunchKernelGGL((attend_many_join_kernel<DIM, BF16>), dim3(static_cast<unsigned>(a.tokens), static_cast<unsigned>(a.heads)),
                     dim3(64), 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace

int64_t many_tiles(const AttendArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.group;
  // every sequence of this kernel has more than few_rows rows, and at most one partial tile
  const int64_t seqs = a.few_rows < 1 ? a.seqs : rows / a.few_rows;
  return rows / kManyRows + (seqs < a.seqs ? seqs : a.seqs);
}

size_t many_part_bytes(const AttendArgs& a) {
  return a.many_splits == 1 ? 0 : static_cast<size_t>(many_tiles(a)) * a.pool.kv_heads * a.many_splits * kManyRows * (a.pool.dim + 2) * 4;
}

hipError_t launch_many(const AttendArgs& given, float* ws) {
  AttendArgs a = given;
  const int64_t grid = many_tiles(a) * a.pool.kv_heads * a.many_splits;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  a.many_part = ws;
  a.many_ml = ws + grid * kManyRows * a.pool.dim;
  const unsigned g = static_cast<unsigned>(grid);
  if (a.pool.dim == 64) return a.bf16 ? launch_many_of<64, true>(a, g) : launch_many_of<64, false>(a, g);
  return a.bf16 ? launch_many_of<128, true>(a, g) : launch_many_of<128, false>(a, g);
}

}  // namespace mxq
