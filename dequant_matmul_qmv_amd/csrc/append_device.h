// Device helpers shared by the appends to the paged caches: where new tokens go,
// and the scheme of 8 bits.
#pragma once

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
template <typename Args>
__device__ __forceinline__ void new_tokens(const Args& a, int s, int& t0, int& n, int& first) {
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
template <typename Args>
__device__ Touched find_block(const Args& a, int unit) {
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

// Keys as they come: pieces of 8 values, nothing done to them.
struct PlainKeys {
  typedef u4 Raw;
  bool wide;
  __device__ __forceinline__ u4 load(const uint16_t* row, int c) const { return load16(row + c * 8, wide); }
  __device__ __forceinline__ u4 finish(u4 raw, int, int) const { return raw; }
};

// The new tokens of one block and kv head into its page: k and v of them in
// registers between the search for their largest and the rounding.  Run by a
// workgroup; `keys` loads pieces of k's rows and finishes them.
template <bool BF16, int kPer, int kAppendThreads, typename Args, typename Keys>
__device__ __forceinline__ void append_page(const Args& a, const Touched& w, int page, int head, int8_t* tile, const Keys& keys) {
  constexpr int kWaves = kAppendThreads / 64;     // kPer: pieces of 8 values a thread
  __shared__ float red[2][kWaves];
  const int dim = a.pool.dim, b = a.pool.block, tid = threadIdx.x;
  const int64_t ph = static_cast<int64_t>(page) * a.pool.kv_heads + head;
  const uint16_t* kx = a.k + head * a.k_head + w.token * a.k_token;
  const uint16_t* vx = a.v + head * a.v_head + w.token * a.v_token;
  int8_t* k = a.pool.k + ph * dim * b;
  int8_t* v = a.pool.v + ph * dim * b;
  // slot: tokens that the block holds already (all before the first new one)
  const int n = w.hi - w.lo, slot = w.lo - w.j * b, cols_log2 = dim == 64 ? 3 : 4, units = n << cols_log2;

  typename Keys::Raw raw[kPer];
  u4 kr[kPer], vr[kPer];
  float km = 0.0f, vm = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int u = tid + j * kAppendThreads, i = u >> cols_log2, c = u & ((1 << cols_log2) - 1);
    raw[j] = typename Keys::Raw{};
    vr[j] = u4{0, 0, 0, 0};
    if (u < units) {
      raw[j] = keys.load(kx + i * a.k_token, c);
      vr[j] = load16(vx + i * a.v_token + c * 8, a.wide);
    }
  }
  const float k_was = slot > 0 ? a.pool.k_scale[ph] : 0.0f, v_was = slot > 0 ? a.pool.v_scale[ph] : 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int u = tid + j * kAppendThreads;
    kr[j] = keys.finish(raw[j], u >> cols_log2, u & ((1 << cols_log2) - 1));
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

}  // namespace

}  // namespace mxq
