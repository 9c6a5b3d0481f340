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

#include "attend_split.h"

namespace mxq {

namespace {

constexpr float kTiny = 1e-30f;

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

namespace {

struct Parts {
  // Four workgroups a compute unit, or two where four would still have three chunks a
  // wave (64 sequences up to 8192 keys: 45 us with four, 48 with two; 8 of 16384: 59
  // and 55; two of 131071: 105 and 101).
  static constexpr int kPerUnit = 4, kLongChunks = 3 * kFewWaves;
  template <int DIM, int MT, int WAVES>
  static hipError_t launch(const AttendArgs& a, unsigned slots) {
    const dim3 grid(slots), block(64 * WAVES);
    if (a.bf16) hipLaunchKernelGGL((attend_few_kernel<DIM, MT, true, WAVES>), grid, block, 0, a.stream, a);
    else hipLaunchKernelGGL((attend_few_kernel<DIM, MT, false, WAVES>), grid, block, 0, a.stream, a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_attend(const AttendArgs& a, const DeviceInfo& dev) { return launch_attend_parts<Parts>(a, dev); }

}  // namespace mxq
