// New keys and values into the 8-bit paged cache.
//
// A block of `block` tokens and one kv head share a scale: largest magnitude /
// 127, codes rint(x / scale).  A block that is continued keeps its scale while
// the new tokens fit under it; where they do not, the scale grows and the codes
// that are there are rescaled by old / new.  Quotients are taken in f64 and
// rounded once to f32, so that the codes do not depend on a divider.
//
// Bound: HBM for prompts (new tokens read, codes written), launch latency for
// single tokens.  One workgroup holds one (touched block, kv head), so no two
// workgroups share a scale and nothing is atomic.  Measured: 256 single tokens of
// 8 heads 6.4 us on the GPU (8.1 with the call), 5 prompts of up to 4096 tokens (22 MB)
// 9.3 us, most of it the chain starts - table - values - scale.  v is stored
// transposed ([dim, block]): its codes pass through LDS and leave 16 tokens a
// lane; a 16-token piece that also holds older tokens is merged with them.
#include "lanes_device.h"
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

namespace {

struct Touched {
  int seq, j;        // sequence and its block number
  int lo, hi;        // positions [lo, hi) of the new tokens inside this block
  int64_t token;     // row of k and v that holds position lo
  bool any;
};

// New tokens of a sequence: rows [t0, t1), the first at position `first`.
__device__ __forceinline__ void new_tokens(const KvAppendArgs& a, int s, int& t0, int& n, int& first) {
  t0 = min(max(a.starts[s], 0), a.tokens);
  n = min(max(a.starts[s + 1], t0), a.tokens) - t0;
  const int all = max(a.lens[s], 0), len = min(all, a.width * a.pool.block);
  const int over = all - len;        // tokens past the table's last block are dropped
  first = len + over - n;
  if (over > 0) n = max(0, n - over);
  if (first < 0) {                   // more new tokens than the length: the first of them have no place
    n = max(0, n + first);
    t0 -= first;
    first = 0;
  }
}

// The workgroup's block: every wave scans the sequences, 64 at a time.
__device__ Touched find_block(const KvAppendArgs& a, int unit) {
  Touched r{};
  const int b = a.pool.block, lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const int s = s0 + lane;
    int t0 = 0, n = 0, first = 0;
    if (s < a.seqs) new_tokens(a, s, t0, n, first);
    const int count = n > 0 ? (first + n - 1) / b - first / b + 1 : 0;
    const int sum = wave_scan(count);
    const unsigned long long hit = __ballot(before + sum > unit);
    if (hit != 0) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      const int nth = unit - before - (__builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(count, src));
      t0 = __builtin_amdgcn_readlane(t0, src);
      n = __builtin_amdgcn_readlane(n, src);
      first = __builtin_amdgcn_readlane(first, src);
      r.seq = s0 + src;
      r.j = first / b + nth;
      r.lo = max(first, r.j * b);
      r.hi = min(first + n, (r.j + 1) * b);
      r.token = t0 + (r.lo - first);
      r.any = true;
      return r;
    }
    before += last_lane(sum);
  }
  return r;
}

// Eight 16-bit values, as stored.
__device__ __forceinline__ u4 load16(const uint16_t* p, bool wide) {
  if (wide) return *reinterpret_cast<const u4*>(p);
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = static_cast<uint32_t>(p[2 * i]) | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
  return u4{d[0], d[1], d[2], d[3]};
}

// Four codes rescaled.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  int c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = static_cast<int>(__builtin_rintf(static_cast<float>(static_cast<int8_t>(w >> (8 * i))) * ratio));
  return pack_i8x4(c[0], c[1], c[2], c[3]);
}

// The scale with the new tokens' largest magnitude, what older codes are
// multiplied by, and the inverse for new ones.
struct Scaling {
  float now, ratio, inv;
};
__device__ __forceinline__ Scaling scaling(float was, float most) {
  Scaling s{fmaxf(was, static_cast<float>(static_cast<double>(most) / 127.0)), 0.0f, 0.0f};
  if (s.now > 0.0f) {
    s.ratio = static_cast<float>(static_cast<double>(was) / static_cast<double>(s.now));
    s.inv = fminf(static_cast<float>(1.0 / static_cast<double>(s.now)), 3.402823466e38f);
  }
  return s;
}

template <bool BF16>
__device__ __forceinline__ float absmax8(u4 v) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(fabsf(sb_to_f32<BF16>(static_cast<uint16_t>(d[i]))), fabsf(sb_to_f32<BF16>(static_cast<uint16_t>(d[i] >> 16)))));
  return m;
}
template <bool BF16>
__device__ __forceinline__ void quant8(u4 v, float inv, int (&q)[8]) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[2 * i] = quant_i8(sb_to_f32<BF16>(static_cast<uint16_t>(d[i])), inv);
    q[2 * i + 1] = quant_i8(sb_to_f32<BF16>(static_cast<uint16_t>(d[i] >> 16)), inv);
  }
}

}  // namespace

// One new token a sequence: one wave holds a (sequence, kv head), k in its
// first 16 lanes and v in the next, so that both chains of loads run at once
// and no barrier is met.  256 sequences of 8 heads: 2048 waves, one round of
// the chip, where workgroups of 256 threads for each of k and v took two.
template <bool BF16>
__global__ __launch_bounds__(64) void kv_append_one_kernel(KvAppendArgs a) {
  const int seq = blockIdx.x, head = blockIdx.y, lane = threadIdx.x, dim = a.pool.dim, b = a.pool.block;
  const int pos = max(a.lens[seq], 0) - 1;
  if (pos < 0 || pos >= a.width * b) return;
  const int j = pos / b, slot = pos - j * b, c = lane & 15;
  const int page = a.table[static_cast<int64_t>(seq) * a.table_stride + j];
  if (page < 0 || page >= a.pool.blocks) return;  // no such block: the token has no place
  const int64_t ph = static_cast<int64_t>(page) * a.pool.kv_heads + head;
  const bool is_v = (lane & 16) != 0, mine = lane < 32 && c * 8 < dim;
  const uint16_t* x = is_v ? a.v + seq * a.v_token + head * a.v_head : a.k + seq * a.k_token + head * a.k_head;
  float* scale_at = (is_v ? a.pool.v_scale : a.pool.k_scale) + ph;
  const float was = slot > 0 ? *scale_at : 0.0f;
  const u4 raw = mine ? load16(x + c * 8, a.wide) : u4{0, 0, 0, 0};
  float m = absmax8<BF16>(raw);
#pragma unroll
  for (int d = 8; d > 0; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
  const Scaling s = scaling(was, m);
  int8_t* k = a.pool.k + ph * dim * b;
  int8_t* v = a.pool.v + ph * dim * b;
  const float k_ratio = __shfl(s.ratio, 0), v_ratio = __shfl(s.ratio, 16);
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

// Any number of new tokens: one workgroup holds one touched (block, kv head),
// k and v of its new tokens in registers between the search for their largest
// and the rounding.
template <bool BF16, int kPer, int kAppendThreads>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendArgs a) {
  constexpr int kWaves = kAppendThreads / 64;     // kPer: pieces of 8 values a thread
  extern __shared__ __align__(16) int8_t tile[];  // v: [dim][block] codes of the new tokens
  __shared__ float red[2][kWaves];
  const Touched w = find_block(a, blockIdx.x);
  if (!w.any) return;
  const int head = blockIdx.y, dim = a.pool.dim, b = a.pool.block, tid = threadIdx.x;
  const int page = a.table[static_cast<int64_t>(w.seq) * a.table_stride + w.j];
  if (page < 0 || page >= a.pool.blocks) return;  // no such block: the tokens have no place
  const int64_t ph = static_cast<int64_t>(page) * a.pool.kv_heads + head;
  const uint16_t* kx = a.k + head * a.k_head + w.token * a.k_token;
  const uint16_t* vx = a.v + head * a.v_head + w.token * a.v_token;
  int8_t* k = a.pool.k + ph * dim * b;
  int8_t* v = a.pool.v + ph * dim * b;
  // slot: tokens that the block holds already (all before the first new one)
  const int n = w.hi - w.lo, slot = w.lo - w.j * b, cols_log2 = dim == 64 ? 3 : 4, units = n << cols_log2;

  u4 kr[kPer], vr[kPer];
  float km = 0.0f, vm = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int u = tid + j * kAppendThreads, i = u >> cols_log2, c = u & ((1 << cols_log2) - 1);
    kr[j] = vr[j] = u4{0, 0, 0, 0};
    if (u < units) {
      kr[j] = load16(kx + i * a.k_token + c * 8, a.wide);
      vr[j] = load16(vx + i * a.v_token + c * 8, a.wide);
    }
  }
  const float k_was = slot > 0 ? a.pool.k_scale[ph] : 0.0f, v_was = slot > 0 ? a.pool.v_scale[ph] : 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    km = fmaxf(km, absmax8<BF16>(kr[j]));
    vm = fmaxf(vm, absmax8<BF16>(vr[j]));
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    km = fmaxf(km, __shfl_xor(km, d));
    vm = fmaxf(vm, __shfl_xor(vm, d));
  }
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = km;
    red[1][tid >> 6] = vm;
  }
  __syncthreads();  // every thread has read the scales
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    km = fmaxf(km, red[0][i]);
    vm = fmaxf(vm, red[1][i]);
  }
  const Scaling ks = scaling(k_was, km), vs = scaling(v_was, vm);
  if (tid == 0) {
    a.pool.k_scale[ph] = ks.now;
    a.pool.v_scale[ph] = vs.now;
  }
  if (slot > 0 && ks.ratio != 1.0f)
    for (int u = tid; u < slot * dim / 4; u += kAppendThreads) {
      uint32_t* p = reinterpret_cast<uint32_t*>(k) + u;
      *p = rescale4(*p, ks.ratio);
    }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int u = tid + j * kAppendThreads, i = u >> cols_log2, c = u & ((1 << cols_log2) - 1);
    if (u >= units) break;
    int q[8];
    quant8<BF16>(kr[j], ks.inv, q);
    *reinterpret_cast<uint2*>(k + static_cast<int64_t>(slot + i) * dim + c * 8) =
        uint2{pack_i8x4(q[0], q[1], q[2], q[3]), pack_i8x4(q[4], q[5], q[6], q[7])};
    quant8<BF16>(vr[j], vs.inv, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[(c * 8 + e) * b + slot + i] = static_cast<int8_t>(q[e]);
  }
  __syncthreads();
  // pieces of 16 tokens that hold new tokens, or older ones to be rescaled
  const bool rescale = slot > 0 && vs.ratio != 1.0f;
  const int end = slot + n, g0 = rescale ? 0 : slot / 16, g1 = (end + 15) / 16, pieces = g1 - g0;
  for (int u = tid; u < dim * pieces; u += kAppendThreads) {
    const int r = u / pieces, g = g0 + u - r * pieces, at = g * 16;
    u4* p = reinterpret_cast<u4*>(v + static_cast<int64_t>(r) * b + at);
    const u4 fresh = *reinterpret_cast<const u4*>(tile + r * b + at);
    if (at >= slot && at + 16 <= end) {
      *p = fresh;
      continue;
    }
    const u4 old = *p;
    const uint32_t ow[4] = {old.x, old.y, old.z, old.w}, fw[4] = {fresh.x, fresh.y, fresh.z, fresh.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t scaled = rescale ? rescale4(ow[i], vs.ratio) : ow[i];
      o[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int sl = at + i * 4 + e;
        const uint32_t src = sl < slot ? scaled : sl < end ? fw[i] : ow[i];
        o[i] |= src & (0xFFu << (8 * e));
      }
    }
    *p = u4{o[0], o[1], o[2], o[3]};
  }
}

namespace {

template <int PER, int THREADS>
hipError_t launch_pages(const KvAppendArgs& a) {
  const int64_t pages = a.tokens / a.pool.block + 2 * static_cast<int64_t>(a.seqs);
  if (!grid_fits(pages, THREADS)) return kTooLarge;
  const dim3 grid(static_cast<unsigned>(pages), static_cast<unsigned>(a.pool.kv_heads));
  const size_t lds = static_cast<size_t>(a.pool.dim) * a.pool.block;
  if (a.bf16) hipLaunchKernelGGL((kv_append_kernel<true, PER, THREADS>), grid, dim3(THREADS), lds, a.stream, a);
  else hipLaunchKernelGGL((kv_append_kernel<false, PER, THREADS>), grid, dim3(THREADS), lds, a.stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a) {
  if (a.starts == nullptr) {
    const dim3 grid(static_cast<unsigned>(a.seqs), static_cast<unsigned>(a.pool.kv_heads));
    if (a.bf16) hipLaunchKernelGGL((kv_append_one_kernel<true>), grid, dim3(64), 0, a.stream, a);
    else hipLaunchKernelGGL((kv_append_one_kernel<false>), grid, dim3(64), 0, a.stream, a);
    return hipGetLastError();
  }
  switch (a.pool.dim * a.pool.block / 2048) {
    case 8: return launch_pages<4, 512>(a);
    case 4: return launch_pages<4, 256>(a);
    case 2: return launch_pages<2, 256>(a);
    default: return launch_pages<1, 256>(a);
  }
}

}  // namespace mxq
