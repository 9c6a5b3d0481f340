// New keys and values into the 8-bit paged cache.
//
// A block of `block` tokens and one kv head share a scale: largest magnitude /
// 127, codes rint(x / scale).  A block that is continued keeps its scale while
// the new tokens fit under it; where they do not, the scale grows and the codes
// that are there are rescaled by old / new.  Quotients are taken in f64 and
// rounded once to f32, so that the codes do not depend on a divider.
//
// Bound: HBM for prompts (new tokens read, codes written), launch latency for
// single tokens.  One workgroup holds one (touched block, kv head) of k or of v,
// so no two workgroups share a scale and nothing is atomic.  v is stored
// transposed ([dim, block]): its codes pass through LDS and leave 16 tokens a
// lane; a 16-token piece that also holds older tokens is merged with them.
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

namespace {

constexpr int kAppendThreads = 256;

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
  const int len = min(max(a.lens[s], 0), a.width * a.pool.block);
  const int over = a.lens[s] - len;  // tokens past the table's last block are dropped
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
  if (a.starts == nullptr) {
    const int pos = a.lens[unit] - 1;
    r.seq = unit;
    r.any = pos >= 0 && pos < a.width * b;
    r.j = pos / b;
    r.lo = pos;
    r.hi = pos + 1;
    r.token = unit;
    return r;
  }
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const int s = s0 + lane;
    int t0 = 0, n = 0, first = 0;
    if (s < a.seqs) new_tokens(a, s, t0, n, first);
    const int count = n > 0 ? (first + n - 1) / b - first / b + 1 : 0;
    int sum = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const unsigned long long hit = __ballot(before + sum > unit);
    if (hit != 0) {
      const int src = __ffsll(hit) - 1;
      const int nth = unit - before - (__shfl(sum, src) - __shfl(count, src));
      t0 = __shfl(t0, src);
      n = __shfl(n, src);
      first = __shfl(first, src);
      r.seq = s0 + src;
      r.j = first / b + nth;
      r.lo = max(first, r.j * b);
      r.hi = min(first + n, (r.j + 1) * b);
      r.token = t0 + (r.lo - first);
      r.any = true;
      return r;
    }
    before += __shfl(sum, 63);
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ void load8(const uint16_t* p, bool wide, float (&f)[8]) {
  uint16_t h[8];
  if (wide) {
    const u4 v = *reinterpret_cast<const u4*>(p);
    __builtin_memcpy(h, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = sb_to_f32<BF16>(h[i]);
}

// Largest over the workgroup.
__device__ __forceinline__ float block_max(float m, float* red) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// Four codes rescaled: those of `mask` bytes only.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  int c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = static_cast<int>(__builtin_rintf(static_cast<float>(static_cast<int8_t>(w >> (8 * i))) * ratio));
  return pack_i8x4(c[0], c[1], c[2], c[3]);
}

}  // namespace

template <bool BF16>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendArgs a) {
  extern __shared__ __align__(16) int8_t tile[];  // v: [dim][block] codes of the new tokens
  __shared__ float red[4];
  const Touched w = find_block(a, blockIdx.x);
  if (!w.any) return;
  const int head = blockIdx.y, dim = a.pool.dim, b = a.pool.block;
  const int page = a.table[static_cast<int64_t>(w.seq) * a.table_stride + w.j];
  if (page < 0 || page >= a.pool.blocks) return;  // no such block: the tokens have no place
  const bool is_v = blockIdx.z != 0;
  const int64_t ph = static_cast<int64_t>(page) * a.pool.kv_heads + head;
  const int64_t ts = is_v ? a.v_token : a.k_token;
  const uint16_t* x = (is_v ? a.v + head * a.v_head : a.k + head * a.k_head) + w.token * ts;
  float* scale_at = (is_v ? a.pool.v_scale : a.pool.k_scale) + ph;
  int8_t* codes = (is_v ? a.pool.v : a.pool.k) + ph * dim * b;
  const int n = w.hi - w.lo, slot = w.lo - w.j * b, cols = dim / 8, units = n * cols;
  // held: tokens that the block holds already (all before the first new one)
  const int held = slot;

  float m = 0.0f;
  for (int u = threadIdx.x; u < units; u += kAppendThreads) {
    const int i = u / cols, c = u - i * cols;
    float f[8];
    load8<BF16>(x + i * ts + c * 8, a.wide, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
  }
  const float was = held > 0 ? *scale_at : 0.0f;
  m = block_max(m, red);  // every thread has read `was` past its barrier
  const float now = fmaxf(was, static_cast<float>(static_cast<double>(m) / 127.0));
  float ratio = 0.0f, inv = 0.0f;
  if (now > 0.0f) {
    ratio = static_cast<float>(static_cast<double>(was) / static_cast<double>(now));
    inv = fminf(static_cast<float>(1.0 / static_cast<double>(now)), 3.402823466e38f);
  }
  if (threadIdx.x == 0) *scale_at = now;
  const bool rescale = held > 0 && ratio != 1.0f;

  if (!is_v) {
    if (rescale)
      for (int u = threadIdx.x; u < held * dim / 4; u += kAppendThreads) {
        uint32_t* p = reinterpret_cast<uint32_t*>(codes) + u;
        *p = rescale4(*p, ratio);
      }
    for (int u = threadIdx.x; u < units; u += kAppendThreads) {
      const int i = u / cols, c = u - i * cols;
      float f[8];
      load8<BF16>(x + i * ts + c * 8, a.wide, f);
      int q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = quant_i8(f[e], inv);
      uint32_t* o = reinterpret_cast<uint32_t*>(codes + static_cast<int64_t>(slot + i) * dim + c * 8);
      o[0] = pack_i8x4(q[0], q[1], q[2], q[3]);
      o[1] = pack_i8x4(q[4], q[5], q[6], q[7]);
    }
    return;
  }

  if (n == 1 && !rescale) {  // one token under the scale that is there: single bytes
    for (int c = threadIdx.x; c < cols; c += kAppendThreads) {
      float f[8];
      load8<BF16>(x + c * 8, a.wide, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) codes[static_cast<int64_t>(c * 8 + e) * b + slot] = static_cast<int8_t>(quant_i8(f[e], inv));
    }
    return;
  }
  for (int u = threadIdx.x; u < units; u += kAppendThreads) {
    const int i = u / cols, c = u - i * cols;
    float f[8];
    load8<BF16>(x + i * ts + c * 8, a.wide, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[(c * 8 + e) * b + slot + i] = static_cast<int8_t>(quant_i8(f[e], inv));
  }
  __syncthreads();
  // pieces of 16 tokens that hold new tokens, or older ones to be rescaled
  const int end = slot + n, g0 = rescale ? 0 : slot / 16, g1 = (end + 15) / 16, pieces = g1 - g0;
  for (int u = threadIdx.x; u < dim * pieces; u += kAppendThreads) {
    const int r = u / pieces, g = g0 + u - r * pieces, at = g * 16;
    u4* p = reinterpret_cast<u4*>(codes + static_cast<int64_t>(r) * b + at);
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
      const uint32_t scaled = rescale ? rescale4(ow[i], ratio) : ow[i];
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

hipError_t launch_kv_append(const KvAppendArgs& a) {
  const int64_t units = a.starts == nullptr ? a.seqs : a.tokens / a.pool.block + 2 * static_cast<int64_t>(a.seqs);
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(a.pool.kv_heads), 2), block(kAppendThreads);
  const size_t lds = static_cast<size_t>(a.pool.dim) * a.pool.block;
  if (a.bf16) hipLaunchKernelGGL((kv_append_kernel<true>), grid, block, lds, a.stream, a);
  else hipLaunchKernelGGL((kv_append_kernel<false>), grid, block, lds, a.stream, a);
  return hipGetLastError();
}

}  // namespace mxq
