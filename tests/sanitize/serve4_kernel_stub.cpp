// Host-only stand-ins for the launch functions behind serve4_api.cpp, for the
// sanitizer build of that layer: as in serve_kernel_stub.cpp, each touches the ends
// (and one byte per 4 KiB) of every range that the real kernels may read or write,
// computed from its arguments.
#include <cstdint>
#include <cstdlib>

#include "serve_internal.h"

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
template <typename F>
void each_row(int64_t tokens, int heads, int64_t token, int64_t head, F f) {
  for (int64_t t = 0; t < tokens; ++t)
    for (int h = 0; h < heads; ++h) f(t * token + h * head);
}
void touch_turn(const mxq::TurnArgs& t, int64_t tokens, int dim) {
  const size_t half = static_cast<size_t>(t.rot / 2), weight = t.weight_f32 ? 4 : 2;
  if (half > 0) touch(t.inv_freq, 4 * half);
  if (half > 0 && t.positions != nullptr)
    for (int a = 0; a < t.axes; ++a) touch(t.positions + a * t.axis_stride, 4 * static_cast<size_t>(tokens));
  if (t.axis != nullptr) touch(t.axis, 4 * half);
  for (const void* w : t.weight)
    if (w != nullptr) touch(w, weight * static_cast<size_t>(dim));
  if (t.axes < 1 || t.rot % 2 != 0 || t.rot > dim) std::abort();
}
void touch_side(const mxq::RopeSide& s, int64_t tokens, int dim) {
  each_row(tokens, s.heads, s.in_token, s.in_head, [&](int64_t at) { touch(s.in + at, 2 * static_cast<size_t>(dim)); });
  each_row(tokens, s.heads, s.out_token, s.out_head, [&](int64_t at) { touch_w(s.out + at, 2 * static_cast<size_t>(dim)); });
}
template <typename Pool>
void touch_pool(const Pool& p, int64_t page, size_t codes, size_t scales) {
  const int64_t head0 = page * p.kv_heads;
  const size_t heads = static_cast<size_t>(p.kv_heads);
  touch_w(reinterpret_cast<char*>(p.k) + head0 * static_cast<int64_t>(codes), codes * heads);
  touch_w(reinterpret_cast<char*>(p.v) + head0 * static_cast<int64_t>(codes), codes * heads);
  touch_w(reinterpret_cast<char*>(p.k_scale) + head0 * static_cast<int64_t>(scales), scales * heads);
  touch_w(reinterpret_cast<char*>(p.v_scale) + head0 * static_cast<int64_t>(scales), scales * heads);
}
size_t codes_of(const mxq::KvPool& p) { return static_cast<size_t>(p.block) * p.dim; }
size_t codes_of(const mxq::KvPool4& p) { return static_cast<size_t>(p.block) * p.dim / 2; }
size_t scales_of(const mxq::KvPool&) { return 4; }
size_t scales_of(const mxq::KvPool4& p) { return 2 * static_cast<size_t>(p.block); }
template <typename Args>
void touch_pages(const Args& a) {
  touch(a.lens, sizeof(int32_t) * static_cast<size_t>(a.seqs));
  if (a.starts) touch(a.starts, sizeof(int32_t) * (static_cast<size_t>(a.seqs) + 1));
  for (int s = 0; s < a.seqs; ++s)
    for (int j = 0; j < a.width; ++j) {
      const int page = a.table[s * a.table_stride + j];
      if (page >= 0 && page < a.pool.blocks) touch_pool(a.pool, page, codes_of(a.pool), scales_of(a.pool));
    }
}
template <typename Args>
hipError_t append(const Args& a) {
  touch_pages(a);
  touch_turn(a.turn, a.tokens, a.pool.dim);
  touch_side(a.q, a.tokens, a.pool.dim);
  each_row(a.tokens, a.pool.kv_heads, a.k_token, a.k_head, [&](int64_t at) { touch(a.k + at, 2 * static_cast<size_t>(a.pool.dim)); });
  each_row(a.tokens, a.pool.kv_heads, a.v_token, a.v_head, [&](int64_t at) { touch(a.v + at, 2 * static_cast<size_t>(a.pool.dim)); });
  if (a.wide && ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) != 0) std::abort();
  if (a.q_wide && ((reinterpret_cast<uintptr_t>(a.q.in) | reinterpret_cast<uintptr_t>(a.q.out)) & 15) != 0) std::abort();
  if (a.q.heads % a.pool.kv_heads != 0) std::abort();
  return hipSuccess;
}

}  // namespace

namespace mxq {

hipError_t launch_norm_rope(const NormRopeArgs& a) {
  touch_turn(a.turn, a.tokens, a.dim);
  for (const RopeSide& s : a.side) touch_side(s, a.tokens, a.dim);
  return hipSuccess;
}
hipError_t launch_rope_append(const RopeAppendArgs& a) { return append(a); }
hipError_t launch_rope_append4(const RopeAppend4Args& a) { return append(a); }

hipError_t launch_attend4(const Attend4Args& a, const DeviceInfo& dev) {
  touch_pages(a);
  each_row(a.tokens, a.heads, a.q_token, a.q_head, [&](int64_t at) { touch(a.q + at, 2 * static_cast<size_t>(a.pool.dim)); });
  const size_t rows = static_cast<size_t>(a.tokens) * a.heads;
  touch_w(a.out, rows * a.pool.dim * 2);
  if (a.lse) touch_w(a.lse, rows * 4);
  if (a.group * a.pool.kv_heads != a.heads) std::abort();
  return with_split_workspace(dev, a.stream, rows * (a.pool.dim + 2) * 4, [&](float* ws) {
    touch_w(ws, rows * (a.pool.dim + 2) * 4);
    return hipSuccess;
  });
}

}  // namespace mxq
