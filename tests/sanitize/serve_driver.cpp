// Driver for the sanitizer build of the serving operators' C-ABI layer
// (serve_api.cpp, with api.cpp and workspace.cpp): every entry point over a
// spread of shapes, types, strides and settings on exact-size host buffers, one
// bad argument at a time, sizes at the ends of their types, and a workspace that
// cannot be had.  Exits 0 and prints "serve sanitize driver: ok" when every
// check holds; a sanitizer report ends the process with an error first.
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

void rope(int64_t tokens, int heads, int kv, int dim, int rot, int inter, mxq_dtype t) {
  // q and k as views of one buffer of [tokens, heads + kv, dim]
  const int64_t row = static_cast<int64_t>(heads + kv) * dim;
  Buf in(static_cast<size_t>(tokens * row * 2)), out(static_cast<size_t>(tokens * row * 2)), f(4u * (rot / 2)), pos(4u * tokens);
  uint16_t *x = in.as<uint16_t>(), *y = out.as<uint16_t>();
  const auto call = [&](uint16_t* q, uint16_t* qo) {
    return mxq_rope(heads ? q : nullptr, row, dim, kv ? q + heads * dim : nullptr, row, dim, heads ? qo : nullptr, row, dim,
                    kv ? qo + heads * dim : nullptr, row, dim, f.as<float>(), pos.as<int32_t>(), tokens, heads, kv, dim, rot, inter, t, kStream);
  };
  CHECK(call(x, y) == MXQ_OK);
  CHECK(call(x, x) == MXQ_OK);
}

struct Paged {
  mxq_kv_cache c{};
  Buf k, v, ks, vs, table, lens, starts, x, y, lse;
  int64_t seqs, width, tokens;
  int heads;
  Paged(int64_t blocks, int kv, int group, int block, int dim, std::vector<int> news, int64_t w)
      : k(static_cast<size_t>(blocks * kv * block * dim)), v(static_cast<size_t>(blocks * kv * block * dim)),
        ks(static_cast<size_t>(blocks * kv * 4)), vs(static_cast<size_t>(blocks * kv * 4)), table(news.size() * w * 4), lens(news.size() * 4),
        starts((news.size() + 1) * 4), x(total(news) * static_cast<size_t>(kv * group * dim) * 2),
        y(total(news) * static_cast<size_t>(kv * group * dim) * 2), lse(total(news) * static_cast<size_t>(kv * group) * 4),
        seqs(static_cast<int64_t>(news.size())), width(w), tokens(static_cast<int64_t>(total(news))), heads(kv * group) {
    c = mxq_kv_cache{k.as<int8_t>(), v.as<int8_t>(), ks.as<float>(), vs.as<float>(), blocks, kv, block, dim};
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

void paged(const Paged& p, bool ragged, mxq_dtype t) {
  const int32_t* st = ragged ? p.starts.as<int32_t>() : nullptr;
  const int64_t qt = static_cast<int64_t>(p.heads) * p.c.dim;
  // k and v: the first kv heads of q's buffer
  CHECK(mxq_kv_append(&p.c, p.x.p, qt, p.c.dim, p.x.p, qt, p.c.dim, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st,
                      p.tokens, p.seqs, t, kStream) == MXQ_OK);
  for (int64_t window : {int64_t{0}, int64_t{9}, kMax64})
    for (float* lse : {static_cast<float*>(nullptr), p.lse.as<float>()})
      CHECK(mxq_attention(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens, p.seqs,
                          p.heads, window, 0.1f, p.y.p, lse, t, kStream) == MXQ_OK);
  // sizes at the ends of their types
  for (int64_t bad : {int64_t{-1}, kMin64, kMax64, kMax64 / 2, int64_t{1} << 60, (int64_t{1} << 32) + 1}) {
    CHECK(mxq_kv_append(&p.c, p.x.p, qt, p.c.dim, p.x.p, qt, p.c.dim, p.table.as<int32_t>(), kMax64, bad, p.lens.as<int32_t>(), st, p.tokens,
                        p.seqs, t, kStream) != MXQ_OK);
    CHECK(mxq_kv_append(&p.c, p.x.p, qt, p.c.dim, p.x.p, qt, p.c.dim, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(),
                        p.starts.as<int32_t>(), bad, p.seqs, t, kStream) != MXQ_OK);
    CHECK(mxq_attention(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), kMax64, bad, p.lens.as<int32_t>(), st, p.tokens, p.seqs, p.heads, 0,
                        0.1f, p.y.p, nullptr, t, kStream) != MXQ_OK);
    CHECK(mxq_attention(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), p.starts.as<int32_t>(),
                        p.tokens, bad, p.heads, 0, 0.1f, p.y.p, nullptr, t, kStream) != MXQ_OK);
    mxq_kv_cache c = p.c;
    c.blocks = bad;
    CHECK(mxq_kv_append(&c, p.x.p, qt, p.c.dim, p.x.p, qt, p.c.dim, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens,
                        p.seqs, t, kStream) != MXQ_OK);
  }
  for (int bad : {-1, kMinInt, kMaxInt}) {
    CHECK(mxq_attention(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens, p.seqs, bad, 0,
                        0.1f, p.y.p, nullptr, t, kStream) != MXQ_OK);
    for (int32_t mxq_kv_cache::*field : {&mxq_kv_cache::kv_heads, &mxq_kv_cache::block, &mxq_kv_cache::dim}) {
      mxq_kv_cache c = p.c;
      c.*field = bad;
      CHECK(mxq_attention(p.x.p, qt, p.c.dim, &c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens, p.seqs, p.heads,
                          0, 0.1f, p.y.p, nullptr, t, kStream) != MXQ_OK);
    }
  }
  for (float bad : {3.4e38f, -2.4e38f, std::numeric_limits<float>::infinity(), std::nanf("")})
    CHECK(mxq_attention(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens, p.seqs, p.heads, 0,
                        bad, p.y.p, nullptr, t, kStream) == MXQ_ERR_INVALID_ARG);
  CHECK(mxq_release_workspaces() >= 0);
  stub_fail_malloc(1);
  CHECK(mxq_attention(p.x.p, qt, p.c.dim, &p.c, p.table.as<int32_t>(), p.width, p.width, p.lens.as<int32_t>(), st, p.tokens, p.seqs, p.heads, 0, 0.1f,
                      p.y.p, nullptr, t, kStream) == MXQ_ERR_HIP);
  stub_fail_malloc(0);
}

void sample(int64_t rows, int64_t vocab, int64_t stride, mxq_dtype t) {
  const size_t size = t == MXQ_F32 ? 4 : 2, n = static_cast<size_t>(rows);
  Buf x(static_cast<size_t>((rows - 1) * stride + vocab) * size), u(n * 4), temp(n * 4), k(n * 4), p(n * 4), m(n * 4), tok(n * 4), prob(n * 4);
  for (int arrays = 0; arrays < 16; ++arrays) {
    const mxq_sampling s{arrays & 1 ? temp.as<float>() : nullptr, arrays & 2 ? k.as<int32_t>() : nullptr, arrays & 4 ? p.as<float>() : nullptr,
                         arrays & 8 ? m.as<float>() : nullptr, 0.9f, kMinInt, 0.5f, 0.1f};
    CHECK(mxq_sample(x.p, stride, rows, vocab, t, u.as<float>(), &s, tok.as<int32_t>(), prob.as<float>(), kStream) == MXQ_OK);
  }
  const mxq_sampling s{};
  for (int64_t bad : {int64_t{-1}, kMin64, kMax64, (int64_t{1} << 32) + 1}) {
    CHECK(mxq_sample(x.p, stride, bad, vocab, t, u.as<float>(), &s, tok.as<int32_t>(), prob.as<float>(), kStream) != MXQ_OK);
    CHECK(mxq_sample(x.p, stride, rows, bad, t, u.as<float>(), &s, tok.as<int32_t>(), prob.as<float>(), kStream) != MXQ_OK);
  }
  CHECK(mxq_release_workspaces() >= 0);
  stub_fail_malloc(1);
  CHECK(mxq_sample(x.p, stride, rows, vocab, t, u.as<float>(), &s, tok.as<int32_t>(), prob.as<float>(), kStream) == MXQ_ERR_HIP);
  stub_fail_malloc(0);
}

}  // namespace

int main() {
  for (mxq_dtype t : {MXQ_F16, MXQ_BF16}) {
    for (int inter : {0, 1}) {
      rope(1, 1, 0, 2, 2, inter, t);
      rope(7, 0, 2, 33, 32, inter, t);
      rope(13, 5, 1, 64, 16, inter, t);
      rope(3, 4, 2, 256, 256, inter, t);
      rope(3, 4, 2, 128, 0, inter, t);
    }
    Buf b(4096);
    for (int64_t bad : {int64_t{-1}, kMin64, kMax64, int64_t{1} << 31})
      CHECK(mxq_rope(b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.as<float>(), b.as<int32_t>(), bad, 1, 1, 64, 64, 0, t, kStream) != MXQ_OK);
    for (int bad : {-1, kMinInt, kMaxInt}) {
      CHECK(mxq_rope(b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.as<float>(), b.as<int32_t>(), 1, bad, kMaxInt, 64, 64, 0, t, kStream) != MXQ_OK);
      CHECK(mxq_rope(b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.as<float>(), b.as<int32_t>(), 1, 1, 1, bad, 64, 0, t, kStream) != MXQ_OK);
      CHECK(mxq_rope(b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.p, 64, 64, b.as<float>(), b.as<int32_t>(), 1, 1, 1, 64, bad, 0, t, kStream) != MXQ_OK);
    }
    paged(Paged(6, 2, 4, 16, 64, {1, 1, 1}, 3), false, t);
    paged(Paged(6, 2, 4, 16, 64, {1, 1, 1}, 3), true, t);
    paged(Paged(9, 1, 8, 128, 128, {5, 0, 70, 1}, 2), true, t);
    paged(Paged(3, 3, 1, 32, 128, {40}, 5), true, t);
  }
  for (mxq_dtype t : {MXQ_F16, MXQ_BF16, MXQ_F32}) {
    sample(1, 1, 1, t);
    sample(1, 999, -5, t);   // one row: its stride is not used
    sample(5, 1001, 1001, t);
    sample(3, 1001, 1100, t);
  }
  std::printf("serve sanitize driver: ok\n");
  return 0;
}
