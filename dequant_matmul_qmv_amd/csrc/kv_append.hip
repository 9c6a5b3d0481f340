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
#include "append_device.h"

namespace mxq {

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

// Any number of new tokens: one workgroup holds one touched (block, kv head).
template <bool BF16, int kPer, int kAppendThreads>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendArgs a) {
  extern __shared__ __align__(16) int8_t tile[];  // v: [dim][block] codes of the new tokens
  const Touched w = find_block(a, blockIdx.x);
  if (!w.any) return;
  const int page = a.table[static_cast<int64_t>(w.seq) * a.table_stride + w.j];
  if (page < 0 || page >= a.pool.blocks) return;  // no such block: the tokens have no place
  append_page<BF16, kPer, kAppendThreads>(a, w, page, blockIdx.y, tile, PlainKeys{a.wide});
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
