// Attention of a few new tokens a sequence over the 4-bit paged cache: the serving
// step's form (one token), and short drafts.
//
//   x = (q . c - z sum q) * s * scale,  p = exp(x - max x),
//   out = sum p (c' - z') s' / sum p
//
// with c, z, s a key's codes, zero point and scale, c', z', s' a value's; masks as
// for the 8-bit cache.
//
// Bound: HBM, the cache read once (keys * kv heads * (dim + 4) bytes).  The key axis
// is divided over workgroups as there (attend_split.h).
//
// Both products run on the matrix cores straight from registers.  S^T = K Q^T, keys
// as 16 rows, leaves lane group h four keys of one query row in each tile; with the
// rows of two tiles dealt out so that those are the 8 tokens that a word of v holds,
// in the order in which its codes unpack, the weights are the operand of
// O^T = V^T P^T in place.  k's codes go in as f16 subnormals, unscaled: a key's scale
// and zero point are applied to its score.  v's become values, exact in f16.
//
// Rounding: q, keys and values exact; sums, maxima and weights f32; P is f16, held as
// 2^14 times its value (the weights are summed before that rounding).
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
  bool ok[2];               // their page is there
};

struct Pages4 {
  int k[2], v[2];  // pages of the lane's k rows and of its v tokens; -1: none
};

template <int N>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u4 x = *reinterpret_cast<const u4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  }
}

}  // namespace

template <int DIM, int MT, bool BF16, int WAVES>
__global__ __launch_bounds__(64 * WAVES, MT * DIM >= 256 && WAVES == kFewWaves ? 1 : 2) void attend4_few_kernel(Attend4Args a) {
  constexpr int KW = DIM / 32, DP = DIM / 64, kRows = 16 * MT;
  __shared__ float join[WAVES][16][DIM + 4];
  __shared__ float join_m[WAVES][16], join_l[WAVES][16];
  const Part part = find_part<MT>(a, blockIdx.x, -1);
  if (!part.any) return;
  const int hk = a.pool.kv_heads, block = a.pool.block, block_log2 = 31 - __builtin_clz(block);
  const int head = part.nth % hk, rest = part.nth / hk, rg = rest % part.share.groups, split = rest / part.share.groups;
  const SeqSpan sp = seq_span(a, part.seq);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rho = lane & 15, h = lane >> 4;
  const int row0 = rg * kRows, rows = min(kRows, sp.n * a.group - row0);
  const int pos0 = sp.len - sp.n;
  const int limit = min(sp.len, a.width * block);

  // query rows of this lane (one of 16 for each mt): fragments, sums, key ranges
  h8 qf[MT][KW];
  float factor[MT], q_sum[MT];
  int from[MT], upto[MT];
  int all_from = 0, all_upto = INT_MAX;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int i = row0 + mt * 16 + rho;
    const bool real = i < sp.n * a.group;
    const int tok = real ? i / a.group : 0, hq = head * a.group + (real ? i - tok * a.group : 0);
    const uint16_t* q = a.q + static_cast<int64_t>(sp.t0 + tok) * a.q_token + static_cast<int64_t>(hq) * a.q_head;
    u4 raw[KW];
#pragma unroll
    for (int m = 0; m < KW; ++m) raw[m] = *reinterpret_cast<const u4*>(q + h * (DIM / 4) + m * 8);
    float inverse = 1.0f;
    if constexpr (BF16) {
      float top = 0.0f, fac;
#pragma unroll
      for (int m = 0; m < KW; ++m) top = fmaxf(top, absmax8_bf16(raw[m]));
      top = max_xor16(max_xor32(top));
      row_factor(top, fac, inverse);
#pragma unroll
      for (int m = 0; m < KW; ++m) raw[m] = bf16_to_scaled_f16(raw[m], fac);
    }
    factor[mt] = a.scale2 * inverse;
    float sum = 0.0f;
#pragma unroll
    for (int m = 0; m < KW; ++m) {
      sum += sum8_f32(raw[m]);
      qf[mt][m] = as_h8(perm_x_w4(raw[m]));
    }
    q_sum[mt] = add_xor16(add_xor32(sum));
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
  const int k_row = 8 * (rho >> 2) + 4 * (rho & 1) + ((rho >> 1) & 1);  // of 32 keys; 2 more in the second tile

  auto pages_of = [&](int c) {
    Pages4 p;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // (a chunk past the end may lie past 2^31)
      const uint32_t key = static_cast<uint32_t>(c) * kChunk + u * 32, width = a.width;
      const uint32_t jk = (key + 8 * (rho >> 2)) >> block_log2, jv = (key + 8 * h) >> block_log2;
      p.k[u] = jk < width ? table[jk] : -1;
      p.v[u] = jv < width ? table[jv] : -1;
    }
    return p;
  };
  auto load_k = [&](int c, const Pages4& p, Raw4<DIM>& r) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t page = p.k[u] >= 0 && p.k[u] < static_cast<int>(a.pool.blocks) ? p.k[u] : 0;
      const int slot = (c * kChunk + u * 32 + k_row) & (block - 1);
      const uint32_t* kp = a.pool.k + ((page * hk + head) * block + slot) * (DIM / 8) + h * KW;
      load_words<KW>(kp, r.k[2 * u]);
      load_words<KW>(kp + 2 * (DIM / 8), r.k[2 * u + 1]);
    }
  };
  auto load_v = [&](int c, const Pages4& p, Raw4<DIM>& r) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = c * kChunk + u * 32 + 8 * h;
      // a page past the sequence's end may be anyone's, or never written
      r.ok[u] = p.v[u] >= 0 && p.v[u] < static_cast<int>(a.pool.blocks) && key < limit;
      const int64_t ph = static_cast<int64_t>(r.ok[u] ? p.v[u] : 0) * hk + head;
      const int slot = key & (block - 1);
      const uint32_t* vp = a.pool.v + (ph * (block / 8) + slot / 8) * DIM + rho * 4;
#pragma unroll
      for (int d = 0; d < DP; ++d) r.v[u][d] = *reinterpret_cast<const u4*>(vp + d * 64);
      r.ks[u] = *reinterpret_cast<const u4*>(a.pool.k_scale + ph * block + slot);
      r.vs[u] = *reinterpret_cast<const u4*>(a.pool.v_scale + ph * block + slot);
    }
  };

  f4 acc[MT][4 * DP];
  float m[MT], l[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = kNegInf;
    l[mt] = 0.0f;
#pragma unroll
    for (int d = 0; d < 4 * DP; ++d) acc[mt][d] = f4{0, 0, 0, 0};
  }

  // one chunk: as soon as k's registers are free they take the next chunk's
  // rows, and v's do after the second product
  auto step = [&](int c, Raw4<DIM>& r, Pages4& ahead) {
    const bool more = c + WAVES < c_end;
    f4 s[MT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][t] = f4{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const h8 k = codes_tiny(r.k[t][w]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qf[mt][w], s[mt][t], 0, 0, 0);
      }
    }
    if (more) load_k(c + WAVES, ahead, r);
    const bool whole = __all(r.ok[0] && r.ok[1]) && c * kChunk >= all_from && c * kChunk <= all_upto - kChunk;
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u) r.vs[u] = first_words(r.vs[u], r.ok[u] ? min(limit - (c * kChunk + u * 32 + 8 * h), 8) : 0);
    }
    float mx[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) mx[mt] = kNegInf;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u4 w4 = perm_x_w4(r.ks[u]);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // key e of the 8, in codes' order
        const uint32_t pair = w[e >> 1];
        const h2 sc = as_h2(pair & 0x7FF07FF0u);
        const float scale = static_cast<float>(e & 1 ? sc.y : sc.x), zero = static_cast<float>((pair >> (16 * (e & 1))) & 15u);
        const int key = c * kChunk + u * 32 + 8 * h + (e >> 1) + 4 * (e & 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float x = __builtin_fmaf(s[mt][2 * u + (e >> 2)][e & 3], kTinyUnit, -zero * q_sum[mt]) * scale * factor[mt];
          if (!whole) x = r.ok[u] && key >= from[mt] && key < upto[mt] ? x : kNegInf;
          mx[mt] = fmaxf(mx[mt], x);
          s[mt][2 * u + (e >> 2)][e & 3] = x;
        }
      }
    }
    u4 pf[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float now = fmaxf(m[mt], max_xor16(max_xor32(mx[mt])));
      const float ref = now == kNegInf ? 0.0f : now;
      const float alpha = __builtin_amdgcn_exp2f(m[mt] - ref);
      m[mt] = now;
      float sum = 0.0f;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = __builtin_amdgcn_exp2f(s[mt][i >> 2][i & 3] - ref + kLift);
        const float p1 = __builtin_amdgcn_exp2f(s[mt][i >> 2][(i & 3) + 1] - ref + kLift);
        sum += p0 + p1;
        const h2 pk = {static_cast<_Float16>(p0), static_cast<_Float16>(p1)};
        w[i / 2] = as_u32(pk);
      }
      l[mt] = l[mt] * alpha + sum;
      pf[mt][0] = u4{w[0], w[1], w[2], w[3]};
      pf[mt][1] = u4{w[4], w[5], w[6], w[7]};
#pragma unroll
      for (int d = 0; d < 4 * DP; ++d) acc[mt][d] *= alpha;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Scales8 sc = scales8(r.vs[u]);
#pragma unroll
      for (int d = 0; d < DP; ++d) {
        const uint32_t w[4] = {r.v[u][d].x, r.v[u][d].y, r.v[u][d].z, r.v[u][d].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const h8 v = values8(w[e], sc);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[mt][d * 4 + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, as_h8(pf[mt][u]), acc[mt][d * 4 + e], 0, 0, 0);
        }
      }
    }
    if (more) {
      load_v(c + WAVES, ahead, r);
      ahead = pages_of(c + 2 * WAVES);
    }
  };

  int c = c_begin + wave;
  if (c < c_end) {
    Raw4<DIM> raw;
    Pages4 ahead = pages_of(c);
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
    // the product's rows are values 64 d + 4 (4 h + i) + e
#pragma unroll
    for (int d = 0; d < DP; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f4*>(&join[wave][rho][d * 64 + h * 16 + i * 4]) =
            f4{acc[mt][d * 4][i], acc[mt][d * 4 + 1][i], acc[mt][d * 4 + 2][i], acc[mt][d * 4 + 3][i]};
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

namespace {

struct Parts4 {
  template <int DIM, int MT, int WAVES>
  static hipError_t launch(const Attend4Args& a, unsigned slots) {
    const dim3 grid(slots), block(64 * WAVES);
    if (a.bf16) hipLaunchKernelGGL((attend4_few_kernel<DIM, MT, true, WAVES>), grid, block, 0, a.stream, a);
    else hipLaunchKernelGGL((attend4_few_kernel<DIM, MT, false, WAVES>), grid, block, 0, a.stream, a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_attend4(const Attend4Args& a, const DeviceInfo& dev) { return launch_attend_parts<Parts4>(a, dev); }

}  // namespace mxq
