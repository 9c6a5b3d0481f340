// Host-only stand-ins for the serving operators' launch functions, for the
// sanitizer build of their C-ABI layer (serve_api.cpp): as in kernel_stub.cpp,
// each touches the ends (and one byte per 4 KiB) of every range that the real
// kernels may read or write, computed from its arguments.  Lengths, starts and
// tables are host memory here and are read as the kernels read them.
#include <cstdint>
#include <cstdlib>

#include "serve_internal.h"

hipError_t hipMallocAsync(void** p, size_t bytes, hipStream_t) {
  *p = std::malloc(bytes ? bytes : 1);
  return *p == nullptr ? hipErrorOutOfMemory : hipSuccess;
}
hipError_t hipFreeAsync(void* p, hipStream_t) {
  std::free(p);
  return hipSuccess;
}

namespace {

void touch(const void* p, size_t bytes) {
  const volatile unsigned char* c = static_cast<const volatile unsigned char*>(p);
  unsigned char acc = 0;
  for (size_t i = 0; i < bytes; i += 4096) acc ^= c[i];
  if (bytes) acc ^= c[bytes - 1];
  (void)acc;
}
void touch_w(void* p, size_t bytes) {
  volatile unsigned char* c = static_cast<volatile unsigned char*>(p);
  for (size_t i = 0; i < bytes; i += 4096) c[i] = 0;
  if (bytes) c[bytes - 1] = 0;
}
// rows of a [tokens, heads, dim] view
template <typename F>
void each_row(int64_t tokens, int heads, int64_t token, int64_t head, F f) {
  for (int64_t t = 0; t < tokens; ++t)
    for (int h = 0; h < heads; ++h) f(t * token + h * head);
}
// the pages of the sequences' tables that exist
template <typename A, typename F>
void each_page(const A& a, F f) {
  for (int s = 0; s < a.seqs; ++s)
    for (int j = 0; j < a.width; ++j) {
      const int page = a.table[s * a.table_stride + j];
      if (page >= 0 && page < a.pool.blocks) f(static_cast<int64_t>(page) * a.pool.kv_heads);
    }
}
template <typename A>
void touch_lengths(const A& a) {
  touch(a.lens, sizeof(int32_t) * static_cast<size_t>(a.seqs));
  if (a.starts) touch(a.starts, sizeof(int32_t) * (static_cast<size_t>(a.seqs) + 1));
}

}  // namespace

namespace mxq {

hipError_t launch_rope(const RopeArgs& a) {
  touch(a.positions, sizeof(int32_t) * static_cast<size_t>(a.tokens));
  if (a.rot > 0) touch(a.inv_freq, sizeof(float) * static_cast<size_t>(a.rot / 2));
  for (const RopeSide& s : a.side) {
    each_row(a.tokens, s.heads, s.in_token, s.in_head, [&](int64_t at) { touch(s.in + at, 2 * static_cast<size_t>(a.dim)); });
    each_row(a.tokens, s.heads, s.out_token, s.out_head, [&](int64_t at) { touch_w(s.out + at, 2 * static_cast<size_t>(a.dim)); });
  }
  return hipSuccess;
}

hipError_t launch_kv_append(const KvAppendArgs& a) {
  touch_lengths(a);
  each_row(a.tokens, a.pool.kv_heads, a.k_token, a.k_head, [&](int64_t at) { touch(a.k + at, 2 * static_cast<size_t>(a.pool.dim)); });
  each_row(a.tokens, a.pool.kv_heads, a.v_token, a.v_head, [&](int64_t at) { touch(a.v + at, 2 * static_cast<size_t>(a.pool.dim)); });
  each_page(a, [&](int64_t ph) {
    const size_t codes = static_cast<size_t>(a.pool.kv_heads) * a.pool.block * a.pool.dim, heads = static_cast<size_t>(a.pool.kv_heads);
    touch_w(a.pool.k + ph * a.pool.block * a.pool.dim, codes);
    touch_w(a.pool.v + ph * a.pool.block * a.pool.dim, codes);
    touch_w(a.pool.k_scale + ph, 4 * heads);
    touch_w(a.pool.v_scale + ph, 4 * heads);
  });
  if (a.wide && ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) != 0) std::abort();
  return hipSuccess;
}

hipError_t launch_attend(const AttendArgs& a, const DeviceInfo& dev) {
  touch_lengths(a);
  each_row(a.tokens, a.heads, a.q_token, a.q_head, [&](int64_t at) { touch(a.q + at, 2 * static_cast<size_t>(a.pool.dim)); });
  each_page(a, [&](int64_t ph) {
    const size_t codes = static_cast<size_t>(a.pool.kv_heads) * a.pool.block * a.pool.dim, heads = static_cast<size_t>(a.pool.kv_heads);
    touch(a.pool.k + ph * a.pool.block * a.pool.dim, codes);
    touch(a.pool.v + ph * a.pool.block * a.pool.dim, codes);
    touch(a.pool.k_scale + ph, 4 * heads);
    touch(a.pool.v_scale + ph, 4 * heads);
  });
  const size_t rows = static_cast<size_t>(a.tokens) * a.heads;
  touch_w(a.out, rows * a.pool.dim * 2);
  if (a.lse) touch_w(a.lse, rows * 4);
  if (a.group * a.pool.kv_heads != a.heads) std::abort();
  return with_split_workspace(dev, a.stream, rows * (a.pool.dim + 2) * 4, [&](float* ws) {
    touch_w(ws, rows * (a.pool.dim + 2) * 4);
    return hipSuccess;
  });
}

hipError_t launch_sample(const SampleArgs& a, const DeviceInfo& dev) {
  const size_t rows = static_cast<size_t>(a.rows), size = a.type == MXQ_F32 ? 4 : 2;
  for (size_t r = 0; r < rows; ++r) touch(static_cast<const char*>(a.logits) + r * a.row_stride * size, a.vocab * size);
  touch(a.u, rows * 4);
  if (a.temperature) touch(a.temperature, rows * 4);
  if (a.top_k) touch(a.top_k, rows * 4);
  if (a.top_p) touch(a.top_p, rows * 4);
  if (a.min_p) touch(a.min_p, rows * 4);
  touch_w(a.tokens, rows * 4);
  touch_w(a.probs, rows * 4);
  return with_split_workspace(dev, a.stream, rows * 4096, [&](float* ws) {
    touch_w(ws, rows * 4096);
    return hipSuccess;
  });
}

}  // namespace mxq
