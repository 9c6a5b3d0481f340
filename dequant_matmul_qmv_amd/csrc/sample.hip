// Drawing the next token from logits with temperature, top-k, top-p and min-p,
// given a uniform number.
//
// With w_i = exp((x_i - max x) / temperature), the kept tokens are a prefix of
// the descending order (equals by index): at most top_k of them, the shortest
// that reaches top_p of the weight of those, and w_i >= min_p.  The token drawn
// is the first, in index order, whose running sum of kept weights exceeds
// u * their total.
//
// Which token a border falls on is a whole number, so weights are taken in f64.
// Where threads add in no fixed order they add integers of 2^-43: such sums are
// the same in any order, and a border is off by 2^-44 a token of a total that is
// at least 1.  A token below 2^-44 of the largest has the integer 0: where a row
// has limits it can neither be drawn nor move a border, and is left out.  Rows
// without limits add pieces of 512 tokens as integers, the tokens of one piece in
// f64, in a fixed order.
//
// The descending order is that of one number a token, its word: the logit as an
// ordered 32-bit key, then the index, the lower the larger.  Words differ, so a
// prefix is held as its last word, and "kept" is word >= end and weight >= min_p.
//
// Bound: one read of the logits, and one f64 exponential for each of them (16
// operations) where the whole row's weight is asked for.  Four kernels:
//   stats   many workgroups a row: the largest value of each cell of 64 tokens;
//           where no top-k limits the row, also the weight of each piece of 512,
//           relative to the piece's own largest
//   draw    one workgroup a row.  Without limits it adds the pieces, finds the
//           one that u falls in and looks at its tokens alone.  With limits the
//           cells give a bound that no kept token is below (the k-th largest
//           cell bounds the k-th largest token), and only cells that reach it
//           are read again, into a list of at most 2048 tokens in LDS.  Rows
//           whose kept tokens are more than that are left to the last two
//   bins    many workgroups a row: counts and weights of 2048 bins by value.  For
//           few rows these are further workgroups of the draw kernel, which work
//           before it is known whether they are needed
//   wide    many workgroups a row: the bins say in which of them the prefix
//           ends; their tokens go to a list, those before them into the kept
//           weight of their piece.  The row's last workgroup (a fifth kernel where
//           the rows are many) finds the end in
//           the list and draws.  Where a bin has more tokens than a list (many
//           equal logits) it searches the row itself
// Measured: one row of 128256, top-k 40 and top-p, 13.5 .. 15.5 us by card (draw
// 9, stats 2.9), or 36 .. 38 with a prefix of thousands; 192 rows of mixed settings
// 118 us (stats 24, draw 33, bins 22, wide 29, the draw after it 13); 17 rows of
// 32003 by min-p 20 us (draw 16).
// One workgroup a row for everything took 323, 528 and 40 us.
#include <cfloat>

#include "lanes_device.h"
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

namespace {

constexpr int kDrawThreads = 1024, kDrawWaves = 16;
constexpr int kCell = 64, kPiece = 512, kStatTokens = 2048;  // tokens of a cell, a piece, a stats workgroup
constexpr int kList = 2048, kShort = 256, kBins = 2048, kMaxPieces = 2048;
constexpr int kGuess = 192;      // cells that a list for top_p alone is taken from
constexpr int kMostRows = 1024;  // rows of one launch: 52 KB of workspace each at 128256 logits
constexpr double kFix = 8796093022208.0;  // 2^43
constexpr float kDeepest = 30.6f;         // 44 ln 2: a token this many temperatures below the largest has no weight

enum { kF16In = 0, kBF16In = 1, kF32In = 2 };

// NaN counts as -inf, -0 as 0; larger values have larger keys, none is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0xFF800000u;
  if (u == 0x80000000u) u = 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int T>
__device__ __forceinline__ float load_logit(const void* row, int i) {
  if constexpr (T == kF32In) return static_cast<const float*>(row)[i];
  else return sb_to_f32<T == kBF16In>(static_cast<const uint16_t*>(row)[i]);
}

// Keys of 8 tokens from i on; 0 past n.  Rows may start at any element: the
// loads are wide all the same, global memory takes them at any address.
template <int T>
__device__ __forceinline__ void load_keys8(const void* row, int i, int n, uint32_t (&key)[8]) {
  const int at = min(i, max(n - 8, 0));  // a whole piece, or the row's last 8
  if (n >= 8) {
    float f[8];
    if constexpr (T == kF32In) {
      __builtin_memcpy(f, static_cast<const float*>(row) + at, 32);
    } else {
      uint16_t h[8];
      __builtin_memcpy(h, static_cast<const uint16_t*>(row) + at, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = sb_to_f32<T == kBF16In>(h[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) key[e] = key_of(f[e]);
    if (at != i) {  // the first of them belong to the piece before
      const int skip = i - at;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t k = 0;
#pragma unroll
        for (int d = e; d < 8; ++d) k = d == e + skip ? key[d] : k;
        key[e] = k;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) key[e] = i + e < n ? key_of(load_logit<T>(row, min(i + e, n - 1))) : 0;
  }
}

// 2^z for z <= 0: whole part by the exponent, the rest, within a half, by the
// series of exp(r ln 2) to r^11 (6e-15).  0 for -infinity (and NaN: 0 times it,
// a masked token at an infinite temperature).
__device__ __forceinline__ double exp2_neg(double z) {
  z = fmax(z, -1100.0);
  const double n = __builtin_rint(z), r = (z - n) * 0.69314718055994530942;
  double y = 1.0 / 39916800.0;
  y = __builtin_fma(y, r, 1.0 / 3628800.0);
  y = __builtin_fma(y, r, 1.0 / 362880.0);
  y = __builtin_fma(y, r, 1.0 / 40320.0);
  y = __builtin_fma(y, r, 1.0 / 5040.0);
  y = __builtin_fma(y, r, 1.0 / 720.0);
  y = __builtin_fma(y, r, 1.0 / 120.0);
  y = __builtin_fma(y, r, 1.0 / 24.0);
  y = __builtin_fma(y, r, 1.0 / 6.0);
  y = __builtin_fma(y, r, 0.5);
  y = __builtin_fma(y, r, 1.0);
  y = __builtin_fma(y, r, 1.0);
  return ldexp(y, static_cast<int>(n));
}

// Weight of a key relative to `top`, and its integer.
struct Weigh {
  uint32_t top;
  double top_value, per;  // per: log2(e) / temperature
  __device__ __forceinline__ double weight(uint32_t key) const {
    return key == top ? 1.0 : exp2_neg((static_cast<double>(value_of(key)) - top_value) * per);
  }
  // more than 2^-44; key 0 is no token
  __device__ __forceinline__ bool exists(uint32_t key) const {
    return key != 0 && (key == top || (static_cast<double>(value_of(key)) - top_value) * per > -44.0);
  }
  __device__ __forceinline__ u64 fixed(uint32_t key) const {
    return exists(key) ? static_cast<u64>(__builtin_rint(weight(key) * kFix)) : 0;
  }
};
__device__ __forceinline__ Weigh weigher(uint32_t top, float temperature) {
  return Weigh{top, static_cast<double>(value_of(top)), 1.44269504088896340736 / static_cast<double>(temperature)};
}

// A row's settings.
struct Rule {
  float t, p, min_p;
  int k;         // n: no limit
  bool one;      // the largest, the first of equals
  bool open;     // no limit at all
  bool by_piece; // the weight of the whole row is asked for
};
__device__ __forceinline__ Rule rule_of(const SampleArgs& a, int row) {
  Rule r;
  r.t = a.temperature ? a.temperature[row] : a.temperature_all;
  r.p = a.top_p ? a.top_p[row] : a.top_p_all;
  r.min_p = a.min_p ? a.min_p[row] : a.min_p_all;
  r.k = a.top_k ? a.top_k[row] : a.top_k_all;
  r.one = !(r.t > 0.0f) || !(r.p > 0.0f) || !(r.min_p <= 1.0f) || r.k == 1;
  if (r.k <= 0 || r.k > a.vocab) r.k = a.vocab;
  r.open = !r.one && r.k == a.vocab && r.p >= 1.0f && !(r.min_p > 0.0f);
  r.by_piece = !r.one && r.k == a.vocab && (r.p < 1.0f || !(r.min_p > 0.0f));
  return r;
}

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int row, int size) {
  return static_cast<const char*>(a.logits) + static_cast<int64_t>(row) * a.row_stride * size;
}

// The row's uniform number; below 0 as 0, so that every row has a token to draw.
__device__ __forceinline__ double uniform_of(const SampleArgs& a, int row) {
  const float u = a.u[row];
  return u < 0.0f ? 0.0 : static_cast<double>(u);
}

// A token's place in the descending order: its key, equals by index.
__device__ __forceinline__ u64 word_of(uint32_t key, int i) { return (static_cast<u64>(key) << 20) | (0xFFFFFu - static_cast<uint32_t>(i)); }
// The smallest word of a key.
__device__ __forceinline__ u64 first_word(uint32_t key) { return static_cast<u64>(key) << 20; }
__device__ __forceinline__ uint32_t key_in(u64 word) { return static_cast<uint32_t>(word >> 20); }
__device__ __forceinline__ int index_in(u64 word) { return static_cast<int>(0xFFFFFu - (static_cast<uint32_t>(word) & 0xFFFFFu)); }

// A row's state: drawn, or what the last two kernels have to do.
enum { kDone = 0, kSums = 1, kBinned = 2, kSearch = 3 };  // sums alone; a prefix that ends in a bin; a search in the row

// Bins by value: equal widths from the largest down; the last one holds all that is further.
struct Bins {
  float top, scale;
  __device__ __forceinline__ int of(uint32_t key) const {
    const float d = (top - value_of(key)) * scale;
    return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
  }
};

struct Shared {
  u64 word[kList];  // the list
  union {
    struct {
      union {
        u64 mass[kList];
        int hit[kList];  // cells to be read, before the list has weights
      };
      union {
        u64 piece[kMaxPieces];  // kept weight
        struct {
          uint32_t count[256];
          u64 mass[256];
        } digit;
        struct {
          uint32_t rank[4][kShort];
          u64 ahead[4][kShort];
        } pairs;
        uint32_t bin[kBins];
      };
    };
    uint32_t some[kDrawWaves][kPiece];  // keys of a wave's piece
  };
  uint32_t bin_count[kBins];            // beside word, which then holds the bins' weights
  u64 wave_mass[kDrawWaves], wave_bits[kDrawWaves];
  uint32_t wave_count[kDrawWaves], red[kDrawWaves];
  u64 above, end, other;
  uint32_t found, hits, listed;
};
static_assert(kMaxPieces * kPiece == 1 << 20 && kMaxPieces == 2 * kDrawThreads && kBins == 2 * kDrawThreads, "two a thread");

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ u64 block_sum(Shared& sh, u64 x) {
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave_mass[threadIdx.x >> 6] = x;
  __syncthreads();
  u64 s = 0;
  for (int i = 0; i < kDrawWaves; ++i) s += sh.wave_mass[i];
  return s;
}
__device__ __forceinline__ uint32_t block_max(Shared& sh, uint32_t x) {
  x = wave_max(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.red[threadIdx.x >> 6] = x;
  __syncthreads();
  return wave_max(sh.red[threadIdx.x & (kDrawWaves - 1)]);
}

// The word at which the count (or weight) of the larger ones and its own
// reaches `want`, or 0, digit by digit (8 bits) from the first bit in which the
// words differ.  get(i, word, mass) gives item i of `m`, or false; `above` is
// what is larger than all items.
template <typename Get>
__device__ __forceinline__ u64 select_word(Shared& sh, Get get, int m, bool by_mass, double want, u64 above) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  u64 some = 0, any = ~0ull;  // bits set in one of the words, in all of them
#pragma clang loop unroll(disable)
  for (int i = tid; i < m; i += kDrawThreads) {
    u64 word, mass;
    if (!get(i, false, word, mass)) continue;
    some |= word;
    any &= word;
  }
  some = wave_or(some);
  any = ~wave_or(~any);
  __syncthreads();
  if (lane == 0) {
    sh.wave_mass[wave] = some;
    sh.wave_bits[wave] = any;
  }
  __syncthreads();
  for (int i = 0; i < kDrawWaves; ++i) {
    some |= sh.wave_mass[i];
    any &= sh.wave_bits[i];
  }
  if (some == 0) return 0;
  const u64 differ = some & ~any;
  int shift = max(56 - __clzll(differ | 1), 0);  // the first differing bit is the digit's highest
  u64 mask = ~0ull << shift << 8, prefix = some & any & mask;
#pragma clang loop unroll(disable)
  for (;; shift = max(shift - 8, 0)) {
    __syncthreads();
    if (tid < 256) {
      sh.digit.mass[tid] = 0;
      sh.digit.count[tid] = 0;
    }
    if (tid == 0) sh.found = 0;
    __syncthreads();
#pragma clang loop unroll(disable)
    for (int i = tid; i < m; i += kDrawThreads) {
      u64 word, mass;
      if (!get(i, by_mass, word, mass) || (word & mask) != prefix) continue;
      const uint32_t d = static_cast<uint32_t>(word >> shift) & 255u;
      atomicAdd(&sh.digit.count[d], 1u);
      if (by_mass) atomicAdd(&sh.digit.mass[d], mass);
    }
    __syncthreads();
    if (wave == 0) {  // four digits a lane, the largest first
      u64 here[4], sum = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t d = 255u - (lane * 4 + j);
        here[j] = by_mass ? sh.digit.mass[d] : sh.digit.count[d];
        sum += here[j];
      }
      u64 run = above + wave_scan(sum) - sum;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (static_cast<double>(run) < want && static_cast<double>(run + here[j]) >= want) {
          const uint32_t d = 255u - (lane * 4 + j);
          sh.found = d + 1;
          sh.above = run;
          sh.hits = sh.digit.count[d];
        }
        run += here[j];
      }
    }
    __syncthreads();
    if (sh.found == 0) return 0;  // all of them, and less than `want`
    prefix |= static_cast<u64>(sh.found - 1) << shift;
    above = sh.above;
    mask |= 255ull << shift;
    if (shift == 0) return prefix;
    if (sh.hits == 1) {  // it alone
      for (int i = tid; i < m; i += kDrawThreads) {
        u64 word, mass;
        if (get(i, false, word, mass) && (word & mask) == prefix) sh.end = word;
      }
      __syncthreads();
      return sh.end;
    }
  }
}

// Of a wave's 8 keys a lane those that `which` holds for, put side by side into
// its `to` in any order; how many they are.
template <typename Which>
__device__ __forceinline__ int compact(const uint32_t (&key)[8], uint32_t* to, Which which) {
  int held = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool in = which(key[e]);
    const u64 who = __ballot(in);
    if (in) to[held + lanes_below(who)] = key[e];
    held += __popcll(who);
  }
  // the wave's stores before its loads
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return held;
}

// Where u falls: the token drawn is the first, by index, whose sum is over it;
// the last one with weight where u * total reaches the total.
struct Border {
  double target;
  u64 all;
  __device__ __forceinline__ bool over(u64 sum) const {
    return static_cast<double>(all) > target ? static_cast<double>(sum) > target : sum >= all;
  }
};

// The draw among tokens with word >= end and weight >= least: `listed` tokens
// are looked at in the list, the kept weight of all others is in sh.piece.
template <int T>
__device__ __forceinline__ void draw_kept(const SampleArgs& a, Shared& sh, int row, const void* x, const Weigh& w, u64 end,
                                          double least, int listed) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __syncthreads();
  for (int i = tid; i < listed; i += kDrawThreads)
    if (sh.word[i] >= end && static_cast<double>(sh.mass[i]) >= least) atomicAdd(&sh.piece[index_in(sh.word[i]) / kPiece], sh.mass[i]);
  __syncthreads();
  // two pieces a thread, in index order
  const int p = 2 * tid;
  const u64 m0 = p < a.piece_count ? sh.piece[p] : 0, m1 = p + 1 < a.piece_count ? sh.piece[p + 1] : 0;
  const u64 incl = wave_scan(m0 + m1);
  if (lane == 63) sh.wave_mass[wave] = incl;
  __syncthreads();
  u64 base = 0, all = 0;
  for (int i = 0; i < kDrawWaves; ++i) {
    if (i == wave) base = all;
    all += sh.wave_mass[i];
  }
  const Border border{uniform_of(a, row) * static_cast<double>(all), all};
  const auto over = [&](u64 sum) { return border.over(sum); };
  const u64 stop = base + incl, start = stop - m0 - m1;
  if (!over(start) && over(stop)) {
    const bool second = !over(start + m0);
    sh.found = p + (second ? 1 : 0);
    sh.above = second ? start + m0 : start;
  }
  __syncthreads();
  // a token a thread
  const int i = static_cast<int>(sh.found) * kPiece + tid;
  uint32_t key = 0;
  u64 mass = 0;
  if (tid < kPiece && i < a.vocab) {
    key = key_of(load_logit<T>(x, i));
    if (word_of(key, i) >= end) mass = w.fixed(key);
    if (static_cast<double>(mass) < least) mass = 0;
  }
  const u64 sum = wave_scan(mass);
  if (lane == 63) sh.wave_mass[wave] = sum;  // every thread is past its last use
  __syncthreads();
  u64 before = sh.above + sum - mass;
  for (int j = 0; j < wave; ++j) before += sh.wave_mass[j];
  if (mass != 0 && !over(before) && over(before + mass)) {
    a.tokens[row] = i;
    a.probs[row] = static_cast<float>(w.weight(key) * kFix / static_cast<double>(all));
  }
}

// Adds the tokens of part `part` of a row, from `low` up, to the row's bins.
template <int T>
__device__ __forceinline__ void fill_bins(const SampleArgs& a, Shared& sh, int row, const void* x, const Rule& rule, const Weigh& w,
                                          const Bins& bins, uint32_t low, int part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool limit_k = rule.k < a.vocab, limit_p = rule.p < 1.0f;
  u64* mass = sh.word;
  uint32_t* count = sh.bin_count;
  __syncthreads();
  for (int i = tid; i < kBins; i += kDrawThreads) {
    mass[i] = 0;
    count[i] = 0;
  }
  __syncthreads();
  const int upto = min((part + 1) * a.span, a.vocab);
  for (int i = part * a.span + wave * kPiece; i < upto; i += kDrawWaves * kPiece) {
    uint32_t key[8];
    load_keys8<T>(x, i + lane * 8, a.vocab, key);
    // those that can be kept, side by side
    const int held = compact(key, sh.some[wave], [&](uint32_t k) { return k >= low; });
    for (int j = lane; j < held; j += 64) {
      const uint32_t k = sh.some[wave][j];
      const int b = bins.of(k);
      if (limit_k) atomicAdd(&count[b], 1u);
      if (limit_p) atomicAdd(&mass[b], w.fixed(k));
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int i = tid; i < kBins; i += kDrawThreads) {
    if (mass[i] != 0) atomicAdd(&a.bin_mass[static_cast<int64_t>(row) * kBins + i], mass[i]);
    if (count[i] != 0) atomicAdd(&a.bin_count[static_cast<int64_t>(row) * kBins + i], count[i]);
  }
}

// Where the prefix ends, by the bins: the one in which the top_k end, and what
// is before it (kBins: all that is there); top_p of their weight, between that
// without and with this bin, ends in the bins from `first` to `last`.
struct Where {
  int k_bin, first, last;
  u64 k_count, k_mass, first_mass;
};
__device__ __forceinline__ Where locate(const SampleArgs& a, Shared& sh, int row, const Rule& rule, const SamplePlan& plan) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool limit_k = rule.k < a.vocab, limit_p = rule.p < 1.0f;
  const double p = static_cast<double>(rule.p);
  Where at{kBins, kBins, kBins, 0, 0, 0};
  if (plan.state == kBinned) {
    const u64* bin_mass = a.bin_mass + static_cast<int64_t>(row) * kBins;
    const uint32_t* bin_count = a.bin_count + static_cast<int64_t>(row) * kBins;
    const uint32_t c0 = bin_count[2 * tid], c1 = bin_count[2 * tid + 1];
    const u64 m0 = bin_mass[2 * tid], m1 = bin_mass[2 * tid + 1];
    const uint32_t count = wave_scan(c0 + c1);
    const u64 mass = wave_scan(m0 + m1);
    if (lane == 63) {
      sh.wave_count[wave] = count;
      sh.wave_mass[wave] = mass;
    }
    if (tid == 0) sh.found = sh.hits = sh.listed = kBins;
    __syncthreads();
    uint32_t count_base = 0;
    u64 mass_base = 0, all = 0;
    for (int i = 0; i < kDrawWaves; ++i) {
      if (i < wave) count_base += sh.wave_count[i];
      if (i == wave) mass_base = all;
      all += sh.wave_mass[i];
    }
    const uint32_t count_stop = count_base + count, count_start = count_stop - c0 - c1, k = static_cast<uint32_t>(rule.k);
    const u64 mass_stop = mass_base + mass, mass_start = mass_stop - m0 - m1;
    if (limit_k && count_start < k && count_stop >= k) {
      const bool second = count_start + c0 < k;
      sh.found = 2 * tid + (second ? 1 : 0);
      sh.end = second ? count_start + c0 : count_start;
      sh.above = second ? mass_start + m0 : mass_start;
      sh.other = second ? m1 : m0;
    }
    __syncthreads();
    at.k_bin = static_cast<int>(sh.found);
    if (at.k_bin < kBins) {
      at.k_count = sh.end;
      at.k_mass = sh.above;
    } else {
      at.k_mass = all;
    }
    const double least_want = p * (limit_k ? static_cast<double>(at.k_mass) : plan.total);
    const double most_want = limit_k ? p * static_cast<double>(at.k_mass + (at.k_bin < kBins ? sh.other : 0)) : least_want;
    __syncthreads();
    if (limit_p) {
      const auto crosses = [&](double want, u64 from, u64 upto) { return static_cast<double>(from) < want && static_cast<double>(upto) >= want; };
      if (crosses(least_want, mass_start, mass_start + m0)) {
        sh.hits = 2 * tid;
        sh.above = mass_start;
      } else if (crosses(least_want, mass_start + m0, mass_stop)) {
        sh.hits = 2 * tid + 1;
        sh.above = mass_start + m0;
      }
      if (crosses(most_want, mass_start, mass_start + m0)) sh.listed = 2 * tid;
      else if (crosses(most_want, mass_start + m0, mass_stop)) sh.listed = 2 * tid + 1;
      __syncthreads();
      at.first = static_cast<int>(sh.hits);
      at.last = static_cast<int>(sh.listed);
      // not reached: min_p leaves less than top_p does, all that is there is kept; or top_k ends in the first bin
      if (at.first < kBins) at.first_mass = sh.above;
      else if (!(least_want > 0.0)) at.first = 0;
    } else {
      at.first = at.last = at.k_bin;
    }
    __syncthreads();
  }
  return at;
}

// The end of the prefix from the list, or token by token where that is not the
// whole of its bins, and the draw.
template <int T>
__device__ __forceinline__ void finish_row(const SampleArgs& a, Shared& sh, int row, const void* x, const Rule& rule, const Weigh& w,
                                           const Bins& bins, const SamplePlan& plan, const Where& where) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.vocab;
  const bool limit_k = rule.k < n, limit_p = rule.p < 1.0f;
  const double p = static_cast<double>(rule.p);
  const double least = rule.min_p > 0.0f ? static_cast<double>(rule.min_p) * kFix : 0.0;
  const u64* list = a.list + static_cast<int64_t>(row) * kList;
  const u64* kept = a.kept + static_cast<int64_t>(row) * a.piece_count;
  u64 k_mass = where.k_mass;
  if (tid == 0) sh.listed = plan.state == kSearch ? kList + 1 : __hip_atomic_load(&a.plans[row].listed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  int listed = static_cast<int>(sh.listed);
  u64 end = first_word(plan.low);
  if (listed <= kList) {
    for (int i = tid; i < listed; i += kDrawThreads) {
      const u64 word = list[i];
      sh.word[i] = word;
      sh.mass[i] = w.fixed(key_in(word));
    }
    __syncthreads();
    if (where.k_bin < kBins) {
      const auto item = [&](int i, bool, u64& word, u64& mass) {
        word = sh.word[i];
        mass = 0;
        return bins.of(key_in(word)) == where.k_bin;
      };
      end = max(end, select_word(sh, item, listed, false, rule.k, where.k_count));
      u64 held = 0;
      for (int i = tid; i < listed; i += kDrawThreads)
        held += sh.word[i] >= end && bins.of(key_in(sh.word[i])) == where.k_bin ? sh.mass[i] : 0;
      k_mass += block_sum(sh, held);
    }
    if (limit_p && plan.state == kBinned) {
      const auto item = [&](int i, bool, u64& word, u64& mass) {
        word = sh.word[i];
        mass = sh.mass[i];
        return word >= end && bins.of(key_in(word)) <= where.last;
      };
      end = max(end, select_word(sh, item, listed, true, p * (limit_k ? static_cast<double>(k_mass) : plan.total), where.first_mass));
    }
    __syncthreads();
    for (int q = tid; q < a.piece_count; q += kDrawThreads) sh.piece[q] = kept[q];
  } else {
    // the row itself, token by token
    u64 from = 0;
    const auto item = [&](int i, bool weight, u64& word, u64& mass) {
      const uint32_t key = key_of(load_logit<T>(x, i));
      word = word_of(key, i);
      if (key < plan.low || word < from) return false;
      mass = weight ? w.fixed(key) : 0;
      return true;
    };
    listed = 0;
    if (limit_k) {
      from = select_word(sh, item, n, false, rule.k, 0);
      end = max(end, from);
    }
    if (limit_p) {
      double whole = plan.total;
      if (limit_k) {
        u64 held = 0, word, mass;
        for (int i = tid; i < n; i += kDrawThreads) held += item(i, true, word, mass) ? mass : 0;
        whole = static_cast<double>(block_sum(sh, held));
      }
      end = max(end, select_word(sh, item, n, true, p * whole, 0));
    }
    __syncthreads();
    for (int q = wave; q < a.piece_count; q += kDrawWaves) {
      u64 sum = 0;
      for (int i = q * kPiece + lane; i < min((q + 1) * kPiece, n); i += 64) {
        const uint32_t key = key_of(load_logit<T>(x, i));
        const u64 m = word_of(key, i) >= end ? w.fixed(key) : 0;
        sum += static_cast<double>(m) >= least ? m : 0;
      }
      sum = wave_sum(sum);
      if (lane == 0) sh.piece[q] = sum;
    }
  }
  draw_kept<T>(a, sh, row, x, w, end, least, listed);
}

}  // namespace

template <int T>
__global__ __launch_bounds__(256) void sample_stats_kernel(SampleArgs a) {
  const int row = blockIdx.y, lane = threadIdx.x & 63, n = a.vocab;
  const int first = blockIdx.x * kStatTokens + threadIdx.x * 8;
  const void* x = row_of(a, row, T == kF32In ? 4 : 2);
  if (a.ahead)
    for (int i = blockIdx.x * 256 + threadIdx.x; i < kBins; i += gridDim.x * 256) {
      a.bin_mass[static_cast<int64_t>(row) * kBins + i] = 0;
      a.bin_count[static_cast<int64_t>(row) * kBins + i] = 0;
    }
  uint32_t key[8];
  load_keys8<T>(x, first, n, key);
  uint32_t top = key[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) top = max(top, key[e]);
  top = max(top, lane_move<0xB1, 0xF>(top));   // lane ^ 1, ^ 2, and 7 - lane: the same in 8 lanes
  top = max(top, lane_move<0x4E, 0xF>(top));
  top = max(top, lane_move<0x141, 0xF>(top));
  if ((lane & 7) == 0 && first < n) a.cells[static_cast<int64_t>(row) * a.cell_count + first / kCell] = top;
  const Rule r = rule_of(a, row);
  if (!r.by_piece) return;
  top = wave_max(top);
  const Weigh w = weigher(top, r.t);
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += key[e] != 0 ? w.weight(key[e]) : 0.0;
  sum = wave_sum(sum);
  if (lane == 0 && first < n) a.pieces[static_cast<int64_t>(row) * a.piece_count + first / kPiece] = sum;
}

// Where the grid has a second dimension, all but its first workgroups fill the
// row's bins meanwhile: idle compute units' work, which saves a launch (one row:
// 16.0 us with the launch, 13.6 without; a prefix of thousands: 41.7 and 36.5).
template <int T>
__global__ __launch_bounds__(kDrawThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.vocab;
  const void* x = row_of(a, row, T == kF32In ? 4 : 2);
  const uint32_t* cells = a.cells + static_cast<int64_t>(row) * a.cell_count;
  const double* pieces = a.pieces + static_cast<int64_t>(row) * a.piece_count;
  const Rule rule = rule_of(a, row);
  if (blockIdx.y != 0 && (rule.one || rule.open)) return;

  // this thread's cells: the first two in registers
  constexpr int kHeld = 2;
  uint32_t cell[kHeld];
#pragma unroll
  for (int e = 0; e < kHeld; ++e) cell[e] = tid + e * kDrawThreads < a.cell_count ? cells[tid + e * kDrawThreads] : 0;
  auto each_cell = [&](auto f) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e)
      if (tid + e * kDrawThreads < a.cell_count) f(tid + e * kDrawThreads, cell[e]);
    for (int c = tid + kHeld * kDrawThreads; c < a.cell_count; c += kDrawThreads) f(c, cells[c]);
  };
  uint32_t top = 0;
  each_cell([&](int, uint32_t key) { top = max(top, key); });
  if (tid == 0) {
    sh.found = 0x7FFFFFFF;
    sh.hits = sh.listed = 0;
    if (a.plans && blockIdx.y == 0) a.plans[row].state = kDone;
  }
  top = block_max(sh, top);
  const Weigh w = weigher(top, rule.one ? 1.0f : rule.t);

  if (rule.one) {
    each_cell([&](int c, uint32_t key) {
      if (key == top) atomicMin(&sh.found, static_cast<uint32_t>(c));
    });
    __syncthreads();
    if (wave == 0) {
      const int i = static_cast<int>(sh.found) * kCell + lane;
      const u64 hit = __ballot(i < n && key_of(load_logit<T>(x, min(i, n - 1))) == top);
      if (lane == 0) {
        a.tokens[row] = static_cast<int>(sh.found) * kCell + __ffsll(hit) - 1;
        a.probs[row] = 1.0f;
      }
    }
    return;
  }

  // The whole row's weight: that of each piece, rounded to the integers' unit,
  // so that the sums before and through a piece are exact and ascend.
  double total = 0.0;
  const int pieces_each = (a.piece_count + kDrawThreads - 1) / kDrawThreads, p0 = tid * pieces_each;
  u64 piece[2] = {0, 0}, before = 0, all = 0;  // of this thread, before them, of the row
  if (rule.by_piece) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (e < pieces_each && p0 + e < a.piece_count) {
        uint32_t m = 0;
        for (int c = (p0 + e) * (kPiece / kCell); c < min((p0 + e + 1) * (kPiece / kCell), a.cell_count); ++c) m = max(m, cells[c]);
        piece[e] = static_cast<u64>(__builtin_rint(pieces[p0 + e] * w.weight(m) * kFix));
      }
    const u64 incl = wave_scan(piece[0] + piece[1]);
    if (lane == 63) sh.wave_mass[wave] = incl;
    __syncthreads();
    u64 base = 0;
    for (int i = 0; i < kDrawWaves; ++i) {
      if (i == wave) base = all;
      all += sh.wave_mass[i];
    }
    before = base + incl - piece[0] - piece[1];
    total = static_cast<double>(all);
  }

  if (rule.open) {
    // the piece that the border falls in; the last with weight where it reaches the total
    const Border border{uniform_of(a, row) * total, all};
    if (!border.over(before) && border.over(before + piece[0] + piece[1])) {
      const bool second = !border.over(before + piece[0]);
      sh.found = static_cast<uint32_t>(p0) + second;
      sh.above = second ? before + piece[0] : before;
    }
    __syncthreads();
    if (wave != 0) return;
    const int i0 = static_cast<int>(sh.found) * kPiece + lane * 8;
    uint32_t key[8];
    load_keys8<T>(x, i0, n, key);
    double wt[8], s = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wt[e] = key[e] != 0 ? w.weight(key[e]) : 0.0;
      s += wt[e];
    }
    const double incl = static_cast<double>(sh.above) / kFix + wave_scan(s), edge = total > border.target ? border.target / kFix : 1e300;
    const u64 hit = __ballot(incl > edge), some = __ballot(s > 0.0);
    // rounding may leave the tokens' sum a hair short of the piece's: its last token with weight then
    const int src = hit != 0 ? __ffsll(hit) - 1 : 63 - __clzll(some);
    if (lane == src) {
      double run = incl - s;
      int last = 0, pick = -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        run += wt[e];
        if (wt[e] > 0.0) last = e;
        if (pick < 0 && hit != 0 && run > edge && wt[e] > 0.0) pick = e;
      }
      if (pick < 0) pick = last;
      double chosen = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) chosen = e == pick ? wt[e] : chosen;
      a.tokens[row] = i0 + pick;
      a.probs[row] = static_cast<float>(chosen * kFix / total);
    }
    return;
  }

  // A bound that no token with weight is below, then one that no kept token is
  // below: a token is to be listed if its key reaches `low`.
  const float top_x = value_of(top);
  const bool finite = top_x - top_x == 0.0f, limit_k = rule.k < n, limit_p = rule.p < 1.0f, floor = rule.min_p > 0.0f;
  // x >= top - t d, with a margin for its rounding
  auto key_below = [&](double d) {
    const double edge = w.top_value - static_cast<double>(rule.t) * d;
    const double less = edge - 1e-6 * (fabs(edge) + fabs(w.top_value));
    return min(key_of(less > -3.4028e38 ? static_cast<float>(less) : -FLT_MAX), top);
  };
  uint32_t low = finite ? key_below(kDeepest) : top;
  // The cells that hold weight, the furthest of them
  uint32_t far = top;
  each_cell([&](int, uint32_t key) { far = key >= low ? min(far, key) : far; });
  far = ~block_max(sh, ~far);
  const float spread = 2.0f * (top_x - value_of(far)), reach = kDeepest * rule.t;
  const float width = fminf(fmaxf(spread > 0.0f && spread < reach ? spread : reach, 1e-30f), 1e30f);
  const Bins bins{top_x, static_cast<float>(kBins) / width};
  // top_p alone: a list of what is likely; it is no use where it does not hold the whole prefix
  const bool guessed = limit_p && !limit_k && !floor && n > kList;
  // tokens of less than (1 - p) / n of the total: all of them together are less than what top_p leaves out
  if (guessed && finite) low = max(low, key_below(log(static_cast<double>(n) / ((1.0 - static_cast<double>(rule.p)) * (total / kFix)))));
  const uint32_t start = low;
  const bool binned = finite && (limit_k || limit_p);
  const int guess = limit_k ? rule.k : guessed ? min(kGuess, a.cell_count / 2) : 0;
  if (finite && n > kList && guess > 0 && guess <= a.cell_count && guess <= kList) {
    // the guess-th largest cell, to within a bin: at least that many tokens reach its smallest member
    for (int i = tid; i < kBins; i += kDrawThreads) sh.bin[i] = 0;
    __syncthreads();
    each_cell([&](int, uint32_t key) {
      if (key >= low) atomicAdd(&sh.bin[bins.of(key)], 1u);
    });
    if (tid == 0) sh.found = 0;
    __syncthreads();
    const uint32_t b0 = sh.bin[2 * tid], b1 = sh.bin[2 * tid + 1], incl = wave_scan(b0 + b1);
    if (lane == 63) sh.wave_count[wave] = incl;
    __syncthreads();
    uint32_t stop = incl;
    for (int i = 0; i < wave; ++i) stop += sh.wave_count[i];
    const uint32_t want = static_cast<uint32_t>(guess);
    if (stop >= want && stop - b0 - b1 < want) sh.found = 2 * tid + (stop - b1 < want ? 1 : 0) + 1;
    __syncthreads();
    const int bin = static_cast<int>(sh.found) - 1;
    if (bin >= 0) {
      uint32_t least = top;
      each_cell([&](int, uint32_t key) { least = key >= low && bins.of(key) <= bin ? min(least, key) : least; });
      low = ~block_max(sh, ~least);
    }
  }
  // for the row's own kernels; a guess is none
  uint32_t bound = guessed ? start : low;
  // top_p of the top_k needs the weight of all of those, also below min_p
  if (floor && finite && !(limit_k && limit_p)) bound = low = max(low, key_below(-log(static_cast<double>(rule.min_p))));

  if (blockIdx.y != 0) {
    if (binned) fill_bins<T>(a, sh, row, x, rule, w, bins, bound, blockIdx.y - 1);
    return;
  }

  // the list: tokens of `low` and up, from cells that reach it, in no order
  // (more than kList tokens may be kept: not tried)
  if (!limit_k || rule.k <= kList || n <= kList)
    each_cell([&](int c, uint32_t key) {
      if (key >= low) {
        const uint32_t at = atomicAdd(&sh.hits, 1u);
        if (at < kList) sh.hit[at] = c;
      }
    });
  else if (tid == 0)
    sh.hits = kList + 1;
  __syncthreads();
  const int hits = static_cast<int>(sh.hits);
  bool small = hits <= kList;
  if (small) {
    // 8 cells a wave at a time, 8 tokens a lane
#pragma clang loop unroll(disable)
    for (int j = wave * 8; j < hits; j += kDrawWaves * 8) {
      const int h = j + (lane >> 3), first = h < hits ? sh.hit[h] * kCell + (lane & 7) * 8 : n;
      uint32_t key[8], count = 0;
      load_keys8<T>(x, first, n, key);
#pragma unroll
      for (int i = 0; i < 8; ++i) count += key[i] >= low;
      const uint32_t incl = wave_scan(count);
      uint32_t at = 0;
      if (lane == 63) at = atomicAdd(&sh.listed, incl);
      const uint32_t base = last_lane(at);
      if (base > kList) break;  // too many
      at = base + incl - count;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key[i] >= low) {
          if (at < kList) sh.word[at] = word_of(key[i], first + i);
          ++at;
        }
    }
    __syncthreads();
    small = sh.listed <= kList;
  }
  const int listed = static_cast<int>(sh.listed);
  const double least = floor ? static_cast<double>(rule.min_p) * kFix : 0.0;  // of a kept token's integer weight
  u64 end = first_word(low);  // of what is kept; all of the list where nothing limits it further
  if (small) {
    for (int i = tid; i < listed; i += kDrawThreads) sh.mass[i] = w.fixed(key_in(sh.word[i]));
    __syncthreads();
    u64 held = 0;  // the weight of the top_k, or of the list
    if (guessed) {
      for (int i = tid; i < listed; i += kDrawThreads) held += sh.mass[i];
      held = block_sum(sh, held);
      small = static_cast<double>(held) >= static_cast<double>(rule.p) * total;
    }
    if (small && listed <= kShort) {
      // A look from each token at all others, by four threads a token: its
      // place and the weight before it, then the kept weight before it by index.
      const int i = tid & (kShort - 1), team = tid / kShort, share = (listed + 3) / 4;
      const int j0 = team * share, j1 = min(j0 + share, listed);
      const u64 word = i < listed ? sh.word[i] : 0, mass = i < listed ? sh.mass[i] : 0;
      if (i < listed) {
        uint32_t rank = 0;
        u64 ahead = 0;
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
          const bool earlier = sh.word[j] > word;
          rank += earlier;
          ahead += earlier ? sh.mass[j] : 0;
        }
        sh.pairs.rank[team][i] = rank;
        sh.pairs.ahead[team][i] = ahead;
      }
      __syncthreads();
      const bool mine = tid < listed;
      const uint32_t last = static_cast<uint32_t>(min(rule.k, listed)) - 1;
      uint32_t rank = 0;
      u64 ahead = 0;
      if (mine) {
        for (int t = 0; t < 4; ++t) {
          rank += sh.pairs.rank[t][tid];
          ahead += sh.pairs.ahead[t][tid];
        }
        if (rank == last) sh.above = ahead + mass;
      }
      __syncthreads();
      const double want = static_cast<double>(rule.p) * (limit_k ? static_cast<double>(sh.above) : total);
      const bool in = mine && rank <= last && (rank == 0 || !limit_p || static_cast<double>(ahead) < want) &&
                      static_cast<double>(mass) >= least;
      if (mine) sh.mass[tid] = in ? mass : 0;
      __syncthreads();
      if (i < listed) {
        const uint32_t mark = static_cast<uint32_t>(index_in(word));
        u64 sum = 0, all = 0;
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
          const u64 m = sh.mass[j];
          all += m;
          sum += static_cast<uint32_t>(index_in(sh.word[j])) <= mark ? m : 0;
        }
        sh.pairs.ahead[team][i] = sum;
        if (i == 0) sh.wave_mass[team] = all;
      }
      __syncthreads();
      if (!in) return;
      const u64 all = sh.wave_mass[0] + sh.wave_mass[1] + sh.wave_mass[2] + sh.wave_mass[3];
      u64 sum = 0;
      for (int t = 0; t < 4; ++t) sum += sh.pairs.ahead[t][tid];
      const Border border{uniform_of(a, row) * static_cast<double>(all), all};
      if (border.over(sum) && !border.over(sum - mass)) {
        a.tokens[row] = index_in(word);
        a.probs[row] = static_cast<float>(w.weight(key_in(word)) * kFix / static_cast<double>(all));
      }
      return;
    }
    if (small) {
      const auto item = [&](int i, bool, u64& word, u64& mass) {
        word = sh.word[i];
        mass = sh.mass[i];
        return true;
      };
      if (limit_k && rule.k < listed) end = max(end, select_word(sh, item, listed, false, rule.k, 0));
      if (limit_p) {
        if (limit_k) {
          held = 0;
          for (int i = tid; i < listed; i += kDrawThreads) held += sh.word[i] >= end ? sh.mass[i] : 0;
          held = block_sum(sh, held);
        }
        const double want = static_cast<double>(rule.p) * (limit_k ? static_cast<double>(held) : total);
        end = max(end, select_word(sh, item, listed, true, want, 0));
      }
    }
  }
  if (!small) {
    if (tid == 0) {
      const int state = binned ? kBinned : finite && !limit_k && !limit_p ? kSums : kSearch;
      a.plans[row] = SamplePlan{state, top, bound, bins.scale, 0, 0, total};
    }
    if (!a.ahead)
      for (int i = tid; i < kBins; i += kDrawThreads) {
        a.bin_mass[static_cast<int64_t>(row) * kBins + i] = 0;
        a.bin_count[static_cast<int64_t>(row) * kBins + i] = 0;
      }
    return;
  }
  __syncthreads();
  for (int p = tid; p < a.piece_count; p += kDrawThreads) sh.piece[p] = 0;
  draw_kept<T>(a, sh, row, x, w, end, least, listed);
}

template <int T>
__global__ __launch_bounds__(kDrawThreads) void sample_bins_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.y;
  const SamplePlan plan = a.plans[row];
  if (plan.state != kBinned) return;
  const Rule rule = rule_of(a, row);
  fill_bins<T>(a, sh, row, row_of(a, row, T == kF32In ? 4 : 2), rule, weigher(plan.top, rule.t), Bins{value_of(plan.top), plan.scale},
               plan.low, blockIdx.x);
}

// JOINED: the row's last workgroup draws.  Without that the kernel needs few
// registers, and two workgroups fit a compute unit (192 rows: 36 us with both in one).
template <int T, bool JOINED>
__global__ __launch_bounds__(kDrawThreads) void sample_wide_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.vocab;
  const SamplePlan plan = a.plans[row];
  if (plan.state == kDone || (plan.state == kSearch && (blockIdx.x != 0 || !JOINED))) return;
  const void* x = row_of(a, row, T == kF32In ? 4 : 2);
  const Rule rule = rule_of(a, row);
  const Weigh w = weigher(plan.top, rule.t);
  const Bins bins{value_of(plan.top), plan.scale};
  const Where where = locate(a, sh, row, rule, plan);
  if (plan.state != kSearch) {
    const double least = rule.min_p > 0.0f ? static_cast<double>(rule.min_p) * kFix : 0.0;
    u64* list = a.list + static_cast<int64_t>(row) * kList;
    u64* kept = a.kept + static_cast<int64_t>(row) * a.piece_count;
    // a piece a wave at a time
    const int p_end = min((static_cast<int>(blockIdx.x) + 1) * (a.span / kPiece), a.piece_count);
    if (tid == 0) sh.hits = 0;
    __syncthreads();
    for (int q = blockIdx.x * (a.span / kPiece) + wave; q < p_end; q += kDrawWaves) {
      const int i = q * kPiece + lane * 8;
      uint32_t key[8], in_list = 0, sure = 0;
      load_keys8<T>(x, i, n, key);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int b = bins.of(key[e]);
        if (key[e] < plan.low) continue;
        if (b < where.first) sure |= 1u << e;
        else if (b <= where.last || b == where.k_bin) in_list |= 1u << e;
      }
      if (__ballot(in_list != 0) != 0) {
        const uint32_t count = __popc(in_list), incl = wave_scan(count);
        uint32_t at = 0;
        if (lane == 63) at = atomicAdd(&sh.hits, incl);
        at = last_lane(at) + incl - count;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((in_list >> e) & 1u) {
            if (at < kList) sh.word[at] = word_of(key[e], i + e);
            ++at;
          }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) key[e] = (sure >> e) & 1u ? key[e] : 0;
      const int held = compact(key, sh.some[wave], [](uint32_t k) { return k != 0; });
      u64 sum = 0;
      for (int j = lane; j < held; j += 64) {
        const u64 m = w.fixed(sh.some[wave][j]);
        sum += static_cast<double>(m) >= least ? m : 0;
      }
      sum = wave_sum(sum);
      if (lane == 0) kept[q] = sum;
      __builtin_amdgcn_wave_barrier();
    }
    // this workgroup's part of the list
    __syncthreads();
    const uint32_t own = sh.hits;
    if (tid == 0 && own != 0) sh.found = atomicAdd(&a.plans[row].listed, own);
    __syncthreads();
    for (uint32_t i = tid; i < min(own, static_cast<uint32_t>(kList)); i += kDrawThreads)
      if (sh.found + i < kList) list[sh.found + i] = sh.word[i];
    if constexpr (!JOINED) return;
    // The row's last workgroup goes on, with what all have written.  Every wave
    // waits for its own stores to be in the L2 (the barrier does not), then one of
    // them writes that back for the other dies: 8 rows of a long prefix 42 us, 58
    // with a release of the whole in each of the 16 waves.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) sh.found = __hip_atomic_fetch_add(&a.plans[row].arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (sh.found + 1 != gridDim.x) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  }
  if constexpr (JOINED) finish_row<T>(a, sh, row, x, rule, w, bins, plan, where);
}

template <int T>
__global__ __launch_bounds__(kDrawThreads) void sample_finish_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.x;
  const SamplePlan plan = a.plans[row];
  if (plan.state == kDone) return;
  const Rule rule = rule_of(a, row);
  const Weigh w = weigher(plan.top, rule.t);
  const Bins bins{value_of(plan.top), plan.scale};
  const Where where = locate(a, sh, row, rule, plan);
  finish_row<T>(a, sh, row, row_of(a, row, T == kF32In ? 4 : 2), rule, w, bins, plan, where);
}

namespace {

// A row's workspace.
struct Places {
  size_t plans, bin_mass, list, kept, pieces, bin_count, cells, all;
};
Places places_of(const SampleArgs& a, int64_t rows, bool wide) {
  Places p{};
  const auto take = [&](size_t each) {
    const size_t at = p.all;
    p.all += (each * static_cast<size_t>(rows) + 255) / 256 * 256;
    return at;
  };
  p.pieces = take(sizeof(double) * a.piece_count);
  p.cells = take(sizeof(uint32_t) * a.cell_count);
  if (wide) {
    p.plans = take(sizeof(SamplePlan));
    p.bin_mass = take(sizeof(u64) * kBins);
    p.bin_count = take(sizeof(uint32_t) * kBins);
    p.list = take(sizeof(u64) * kList);
    p.kept = take(sizeof(u64) * a.piece_count);
  }
  return p;
}

template <int T>
hipError_t launch_sample_type(const SampleArgs& a, int64_t most_rows, bool wide, int num_cu) {
  for (int64_t r0 = 0; r0 < a.rows; r0 += most_rows) {
    SampleArgs b = a;
    const int rows = static_cast<int>(a.rows - r0 < most_rows ? a.rows - r0 : most_rows);
    b.rows = rows;
    b.logits = static_cast<const char*>(a.logits) + r0 * a.row_stride * (T == kF32In ? 4 : 2);
    b.u += r0;
    if (b.temperature) b.temperature += r0;
    if (b.top_k) b.top_k += r0;
    if (b.top_p) b.top_p += r0;
    if (b.min_p) b.min_p += r0;
    b.tokens += r0;
    b.probs += r0;
    // a row in as many parts as give each compute unit eight workgroups, of 8 tokens a thread at least
    int64_t spans = 8 * num_cu / rows;
    if (spans < 1) spans = 1;
    const int64_t least = kDrawThreads * 8, each = ((a.vocab + spans - 1) / spans + least - 1) / least * least;
    b.span = static_cast<int>(each);
    const dim3 grid(static_cast<unsigned>((a.vocab + each - 1) / each), static_cast<unsigned>(rows));
    // a last workgroup has to wait for its caches' write-back: less than a launch for few of them, more for many
    const bool joined = static_cast<int64_t>(grid.x) * rows <= num_cu;
    b.ahead = wide && joined;
    const unsigned parts = static_cast<unsigned>((a.vocab + kStatTokens - 1) / kStatTokens);
    hipLaunchKernelGGL(sample_stats_kernel<T>, dim3(parts, static_cast<unsigned>(rows)), dim3(256), 0, a.stream, b);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_draw_kernel<T>, dim3(static_cast<unsigned>(rows), b.ahead ? 1 + grid.x : 1), dim3(kDrawThreads), 0, a.stream, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!wide) continue;
    if (joined) {
      hipLaunchKernelGGL((sample_wide_kernel<T, true>), grid, dim3(kDrawThreads), 0, a.stream, b);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      continue;
    }
    hipLaunchKernelGGL(sample_bins_kernel<T>, grid, dim3(kDrawThreads), 0, a.stream, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((sample_wide_kernel<T, false>), grid, dim3(kDrawThreads), 0, a.stream, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_finish_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(kDrawThreads), 0, a.stream, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& given, const DeviceInfo& dev) {
  SampleArgs a = given;
  a.cell_count = (a.vocab + kCell - 1) / kCell;
  a.piece_count = (a.vocab + kPiece - 1) / kPiece;
  // a row longer than a list may need the last two kernels, unless its settings are known here and ask for no prefix
  const bool all_one = (!a.temperature && !(a.temperature_all > 0.0f)) || (!a.top_p && !(a.top_p_all > 0.0f)) ||
                       (!a.min_p && !(a.min_p_all <= 1.0f)) || (!a.top_k && a.top_k_all == 1);
  const bool all_open = !a.top_k && (a.top_k_all <= 0 || a.top_k_all >= a.vocab) && !a.top_p && a.top_p_all >= 1.0f && !a.min_p &&
                        !(a.min_p_all > 0.0f);
  const bool wide = a.vocab > kList && !all_one && !all_open;
  const int64_t held = a.rows < kMostRows ? a.rows : kMostRows;
  const Places at = places_of(a, held, wide);
  return with_split_workspace(dev, a.stream, at.all, [&](float* ws) {
    char* base = reinterpret_cast<char*>(ws);
    a.pieces = reinterpret_cast<double*>(base + at.pieces);
    a.cells = reinterpret_cast<uint32_t*>(base + at.cells);
    if (wide) {
      a.plans = reinterpret_cast<SamplePlan*>(base + at.plans);
      a.bin_mass = reinterpret_cast<u64*>(base + at.bin_mass);
      a.bin_count = reinterpret_cast<uint32_t*>(base + at.bin_count);
      a.list = reinterpret_cast<u64*>(base + at.list);
      a.kept = reinterpret_cast<u64*>(base + at.kept);
    }
    if (a.type == kF16In) return launch_sample_type<kF16In>(a, held, wide, dev.num_cu);
    if (a.type == kBF16In) return launch_sample_type<kBF16In>(a, held, wide, dev.num_cu);
    return launch_sample_type<kF32In>(a, held, wide, dev.num_cu);
  });
}

}  // namespace mxq
