// Driver for the sanitizer build of serve4_api.cpp (with api.cpp and workspace.cpp):
// every entry point over a spread of shapes, types, rotations and strides on
// exact-size host buffers, one bad argument at a time, sizes at the ends of their
// types, and a workspace that cannot be had.  Exits 0 and prints "serve4 sanitize
// driver: ok" when every check holds; a sanitizer report ends the process first.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <vector>

#include "mxq.h"

extern "C" void stub_fail_malloc(int on);

#define CHECK(c)                                                                                 \
  do {                                                                                           \
    if (!(c)) {                                                                                  \
      std::fprintf(stderr, "CHECK failed at %s:%d: %s (last error: %s)\n", __FILE__, __LINE__, #c, \
                   mxq_last_error());                                                            \
      std::exit(1);                                                                              \
    }                                                                                            \
  } while (0)

namespace {

// an exact-size, 256-byte aligned host allocation
struct Buf {
  void* p = nullptr;
  explicit Buf(size_t n) {
    if (posix_memalign(&p, 256, n ? n : 1) != 0) std::abort();
  }
  ~Buf() { std::free(p); }
  Buf(const Buf&) = delete;
  Buf& operator=(const Buf&) = delete;
  template <typename T>
  T* as() const { return static_cast<T*>(p); }
};

void* const kStream = reinterpret_cast<void*>(0x1040);
constexpr int64_t kMax64 = std::numeric_limits<int64_t>::max(), kMin64 = std::numeric_limits<int64_t>::min();
constexpr int kMaxInt = std::numeric_limits<int>::max(), kMinInt = std::numeric_limits<int>::min();

struct Rotation {
  Buf f, pos, axis, qw, kw;
  mxq_rotation r{};
  Rotation(int64_t tokens, int dim, int rot, int axes, mxq_dtype weight, bool places)
      : f(2u * rot), pos(4u * static_cast<size_t>(tokens * axes)), axis(2u * rot), qw(static_cast<size_t>(dim) * (weight == MXQ_F32 ? 4 : 2)),
        kw(static_cast<size_t>(dim) * (weight == MXQ_F32 ? 4 : 2)) {
    r = mxq_rotation{f.as<float>(), places ? nullptr : pos.as<int32_t>(), tokens, axes > 1 ? axis.as<int32_t>() : nullptr, axes, rot, 0, weight,
                     qw.p, kw.p, 1e-6};
  }
};

void norm_rope(int64_t tokens, int heads, int kv, int dim, int rot, int axes, mxq_dtype t, mxq_dtype weight) {
  const int64_t row = static_cast<int64_t>(heads + kv) * dim;
  Buf in(static_cast<size_t>(tokens * row * 2)), out(static_cast<size_t>(tokens * row * 2));
  Rotation rot_(tokens, dim, rot, axes, weight, false);
  uint16_t *x = in.as<uint16_t>(), *y = out.as<uint16_t>();
  const auto call = [&](uint16_t* qo, const mxq_rotation* r) {
    return mxq_norm_rope(heads ? x : nullptr, row, dim, kv ? x + heads * dim : nullptr, row, dim, heads ? qo : nullptr, row, dim,
                         kv ? qo + heads * dim : nullptr, row, dim, r, tokens, heads, kv, dim, t, kStream);
  };
  CHECK(call(y, &rot_.r) == MXQ_OK);
  CHECK(call(x, &rot_.r) == MXQ_OK);
  mxq_rotation r = rot_.r;
  r.q_weight = r.k_weight = nullptr;
  r.weight_dtype = static_cast<mxq_dtype>(3);
  CHECK(call(y, &r) == MXQ_OK);
  r = rot_.r;
  for (int bad : {-1, kMinInt, kMaxInt}) {
    r.rot = bad;
    CHECK(call(y, &r) != MXQ_OK);
    r = rot_.r;
    r.axes = bad;
    CHECK(call(y, &r) != MXQ_OK);
    r = rot_.r;
  }
  for (double bad : {-1e-300, std::numeric_limits<double>::infinity(), std::nan("")}) {
    r.eps = bad;
    CHECK(call(y, &r) == MXQ_ERR_INVALID_ARG);
  }
  r = rot_.r;
  if (axes > 1)
    for (int64_t bad : {tokens - 1, int64_t{-1}, kMin64}) {
      r.position_stride = bad;
      CHECK(call(y, &r) == (rot > 0 ? MXQ_ERR_INVALID_ARG : MXQ_OK));
    }
  for (int64_t bad : {int64_t{-1}, kMin64, kMax64, int64_t{1} << 31})
    CHECK(mxq_norm_rope(x, row, dim, nullptr, 0, 0, y, row, dim, nullptr, 0, 0, &rot_.r, bad, heads, 0, dim, t, kStream) != MXQ_OK);
  for (int bad : {-1, kMinInt, kMaxInt}) {
    CHECK(mxq_norm_rope(x, row, dim, x, row, dim, y, row, dim, y, row, dim, &rot_.r, 1, bad, kMaxInt, dim, t, kStream) != MXQ_OK);
    CHECK(mxq_norm_rope(x, row, dim, x, row, dim, y, row, dim, y, row, dim, &rot_.r, 1, 1, 1, bad, t, kStream) != MXQ_OK);
  }
}

mxq_status append_call(const mxq_kv_cache* c, const void* q, int64_t qt, void* qo, const void* k, const mxq_rotation* r, const int32_t* table,
                       int64_t stride, int64_t width, const int32_t* lens, const int32_t* starts, int64_t tokens, int64_t seqs, int heads,
                       mxq_dtype t) {
  return mxq_rope_append(c, q, qt, c->dim, qo, qt, c->dim, k, qt, c->dim, k, qt, c->dim, r, table, stride, width, lens, starts, tokens, seqs,
                         heads, t, kStream);
}
mxq_status append_call(const mxq_kv_cache4* c, const void* q, int64_t qt, void* qo, const void* k, const mxq_rotation* r, const int32_t* table,
                       int64_t stride, int64_t width, const int32_t* lens, const int32_t* starts, int64_t tokens, int64_t seqs, int heads,
                       mxq_dtype t) {
  return mxq_rope_append4(c, q, qt, c->dim, qo, qt, c->dim, k, qt, c->dim, k, qt, c->dim, r, table, stride, width, lens, starts, tokens, seqs,
                          heads, t, kStream);
}

template <typename Cache>
struct Paged {
  Cache c{};
  Buf k, v, ks, vs, table, lens, starts, x, y, lse;
  int64_t seqs, width, tokens;
  int heads;
  static size_t codes(int64_t n) { return sizeof(*Cache{}.k) == 4 ? static_cast<size_t>(n / 2) : static_cast<size_t>(n); }
  static size_t scales(int64_t pages, int block) { return sizeof(*Cache{}.k) == 4 ? static_cast<size_t>(pages) * block * 2 : static_cast<size_t>(pages) * 4; }
  Paged(int64_t blocks, int kv, int group, int block, int dim, std::vector<int> news, int64_t w)
      : k(codes(blocks * kv * block * dim)), v(codes(blocks * kv * block * dim)), ks(scales(blocks * kv, block)), vs(scales(blocks * kv, block)),
        table(news.size() * w * 4), lens(news.size() * 4), starts((news.size() + 1) * 4), x(total(news) * static_cast<size_t>(kv * group * dim) * 2),
        y(total(news) * static_cast<size_t>(kv * group * dim) * 2), lse(total(news) * static_cast<size_t>(kv * group) * 4),
        seqs(static_cast<int64_t>(news.size())), width(w), tokens(static_cast<int64_t>(total(news))), heads(kv * group) {
    c.k = static_cast<decltype(c.k)>(k.p);
    c.v = static_cast<decltype(c.v)>(v.p);
    c.k_scale = static_cast<decltype(c.k_scale)>(ks.p);
    c.v_scale = static_cast<decltype(c.v_scale)>(vs.p);
    c.blocks = blocks;
    c.kv_heads = kv;
    c.block = block;
    c.dim = dim;
    int at = 0;
    for (size_t s = 0; s < news.size(); ++s) {
      starts.as<int32_t>()[s] = at;
      at += news[s];
      lens.as<int32_t>()[s] = news[s];
      for (int64_t j = 0; j < w; ++j) table.as<int32_t>()[s * w + j] = static_cast<int32_t>((7 * s + 3 * j) % (blocks + 2)) - 1;
    }
    starts.as<int32_t>()[news.size()] = at;
  }
  static size_t total(const std::vector<int>& n) {
    size_t t = 0;
    for (int x : n) t += static_cast<size_t>(x);
    return t;
  }
};

template <typename Cache>
void append(const Paged<Cache>& p, bool ragged, mxq_dtype t) {
  const int32_t* st = ragged ? p.starts.template as<int32_t>() : nullptr;
  const int32_t *tab = p.table.template as<int32_t>(), *len = p.lens.template as<int32_t>();
  const int64_t qt = static_cast<int64_t>(p.heads) * p.c.dim;
  for (int axes : {1, 3})
    for (bool places : {false, true})
      for (int heads : {p.heads, 0}) {
        Rotation r(p.tokens, p.c.dim, p.c.dim / 2, axes, axes == 1 ? t : MXQ_F32, places);
        // k and v: the first kv heads of q's buffer
        CHECK(append_call(&p.c, heads ? p.x.p : nullptr, qt, heads ? p.y.p : nullptr, p.x.p, &r.r, tab, p.width, p.width, len, st, p.tokens, p.seqs,
                          heads, t) == MXQ_OK);
      }
  Rotation r(p.tokens, p.c.dim, p.c.dim, 1, t, false);
  for (int64_t bad : {int64_t{-1}, kMin64, kMax64, kMax64 / 2, int64_t{1} << 60, (int64_t{1} << 32) + 1}) {
    CHECK(append_call(&p.c, p.x.p, qt, p.y.p, p.x.p, &r.r, tab, kMax64, bad, len, st, p.tokens, p.seqs, p.heads, t) != MXQ_OK);
    CHECK(append_call(&p.c, p.x.p, qt, p.y.p, p.x.p, &r.r, tab, p.width, p.width, len, p.starts.template as<int32_t>(), bad, p.seqs, p.heads, t) != MXQ_OK);
    CHECK(append_call(&p.c, p.x.p, qt, p.y.p, p.x.p, &r.r, tab, p.width, p.width, len, p.starts.template as<int32_t>(), p.tokens, bad, p.heads, t) != MXQ_OK);
    Cache c = p.c;
    c.blocks = bad;
    CHECK(append_call(&c, p.x.p, qt, p.y.p, p.x.p, &r.r, tab, p.width, p.width, len, st, p.tokens, p.seqs, p.heads, t) != MXQ_OK);
  }
  for (int bad : {-1, kMinInt, kMaxInt}) {
    CHECK(append_call(&p.c, p.x.p, qt, p.y.p, p.x.p, &r.r, tab, p.width, p.width, len, st, p.tokens, p.seqs, bad, t) != MXQ_OK);
    for (int32_t Cache::*field : {&Cache::kv_heads, &Cache::block, &Cache::dim}) {
      Cache c = p.c;
      c.*field = bad;
      CHECK(append_call(&c, p.x.p, qt, p.y.p, p.x.p, &r.r, tab, p.width, p.width, len, st, p.tokens, p.seqs, p.heads, t) != MXQ_OK);
    }
  }
}

void attention(const Paged<mxq_kv_cache4>& p, bool ragged, mxq_dtype t) {
  const int32_t* st = ragged ? p.starts.as<int32_t>() : nullptr;
  const int64_t qt = static_cast<int64_t>(p.heads) * p.c.dim;
  const auto call = [&](const mxq_kv_cache4& c, int64_t width, int64_t tokens, int64_t seqs, int heads, int64_t window, float scale, float* lse) {
    return mxq_attention4(p.x.p, qt, p.c.dim, &c, p.table.as<int32_t>(), kMax64, width, p.lens.as<int32_t>(), st, tokens, seqs, heads, window, scale,
                          p.y.p, lse, t, kStream);
  };
  const auto good = [&](int64_t window, float* lse) {
    return mxq_attention4(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens, p.seqs, p.heads,
                          window, 0.1f, p.y.p, lse, t, kStream);
  };
  for (int64_t window : {int64_t{0}, int64_t{9}, kMax64})
    for (float* lse : {static_cast<float*>(nullptr), p.lse.as<float>()}) CHECK(good(window, lse) == MXQ_OK);
  CHECK(mxq_kv_append(nullptr, nullptr, 0, 0, nullptr, 0, 0, nullptr, 0, 0, nullptr, nullptr, 0, 0, t, kStream) == MXQ_ERR_INVALID_ARG);
  CHECK(mxq_rope_append4(&p.c, nullptr, 0, 0, nullptr, 0, 0, p.x.p, qt, p.c.dim, p.x.p, qt, p.c.dim, nullptr, p.table.as<int32_t>(), p.width, p.width,
                         p.lens.as<int32_t>(), st, p.tokens, p.seqs, 0, t, kStream) == MXQ_OK);
  for (int64_t bad : {int64_t{-1}, kMin64, kMax64, int64_t{1} << 60, (int64_t{1} << 32) + 1}) {
    CHECK(call(p.c, bad, p.tokens, p.seqs, p.heads, 0, 0.1f, nullptr) != MXQ_OK);
    CHECK(call(p.c, p.width, bad, bad, p.heads, 0, 0.1f, nullptr) != MXQ_OK);
    mxq_kv_cache4 c = p.c;
    c.blocks = bad;
    CHECK(call(c, p.width, p.tokens, p.seqs, p.heads, 0, 0.1f, nullptr) != MXQ_OK);
  }
  for (int bad : {-1, kMinInt, kMaxInt}) CHECK(call(p.c, p.width, p.tokens, p.seqs, bad, 0, 0.1f, nullptr) != MXQ_OK);
  CHECK(call(p.c, p.width, p.tokens, p.seqs, p.heads, -1, 0.1f, nullptr) == MXQ_ERR_INVALID_ARG);
  for (float bad : {3.4e38f, -2.4e38f, std::numeric_limits<float>::infinity(), std::nanf("")})
    CHECK(call(p.c, p.width, p.tokens, p.seqs, p.heads, 0, bad, nullptr) == MXQ_ERR_INVALID_ARG);
  CHECK(mxq_release_workspaces() >= 0);
  stub_fail_malloc(1);
  CHECK(good(0, nullptr) == MXQ_ERR_HIP);
  stub_fail_malloc(0);
}

template <typename F>
void each_paged(mxq_dtype t, F f) {
  f(6, 2, 4, 16, 64, std::vector<int>{1, 1, 1}, 3, false, t);
  f(6, 2, 4, 16, 64, std::vector<int>{1, 1, 1}, 3, true, t);
  f(9, 1, 8, 128, 128, std::vector<int>{5, 0, 70, 1}, 2, true, t);
  f(3, 3, 1, 32, 128, std::vector<int>{40}, 5, true, t);
}

}  // namespace

int main() {
  for (mxq_dtype t : {MXQ_F16, MXQ_BF16}) {
    for (mxq_dtype w : {t, MXQ_F32}) {
      norm_rope(1, 1, 0, 2, 2, 1, t, w);
      norm_rope(7, 0, 2, 33, 32, 2, t, w);
      norm_rope(13, 5, 1, 64, 16, 3, t, w);
      norm_rope(3, 4, 2, 256, 256, 1, t, w);
      norm_rope(3, 4, 2, 128, 0, 2, t, w);
    }
    each_paged(t, [](int64_t blocks, int kv, int group, int block, int dim, const std::vector<int>& news, int64_t w, bool ragged, mxq_dtype type) {
      append(Paged<mxq_kv_cache>(blocks, kv, group, block, dim, news, w), ragged, type);
      append(Paged<mxq_kv_cache4>(blocks, kv, group, block, dim, news, w), ragged, type);
      attention(Paged<mxq_kv_cache4>(blocks, kv, group, block, dim, news, w), ragged, type);
    });
  }
  std::printf("serve4 sanitize driver: ok\n");
  return 0;
}
