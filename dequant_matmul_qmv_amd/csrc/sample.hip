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
// at least 1.  Other sums are f64 in a fixed order.
//
// Bound: one read of the logits, and one f64 exponential for each of them (16
// operations) where the whole row's weight is asked for.  Two kernels:
//   stats   many workgroups a row: the largest value of each cell of 64 tokens;
//           where no top-k limits the row, also the weight of each piece of 512,
//           relative to the piece's own largest
//   draw    one workgroup a row.  Without limits it adds the pieces, finds the
//           one that u falls in and looks at its tokens alone.  With limits the
//           cells give a bound that no kept token is below (the k-th largest
//           cell bounds the k-th largest token), and only cells that reach it are
//           read again: a list of at most 2048 tokens, in LDS, in index order.
//           Rows whose kept tokens are more than that are binned by value, and
//           the bin in which the prefix ends becomes the list.
// A prefix is held as (key, ties): the value at its end, as an ordered 32-bit
// key, and how many of the tokens equal to it belong to it, the first by index.
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

namespace {

constexpr int kDrawThreads = 1024, kDrawWaves = 16;
constexpr int kCell = 64, kPiece = 512, kStatTokens = 2048;  // tokens of a cell, a piece, a stats workgroup
constexpr int kList = 2048, kShort = 256, kBins = 2048;
constexpr double kFix = 8796093022208.0;  // 2^43
typedef unsigned long long u64;

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

// Keys of 8 tokens from i on; 0 past n.  `wide`: they are 16-byte aligned.
template <int T>
__device__ __forceinline__ void load_keys8(const void* row, int i, int n, bool wide, uint32_t (&key)[8]) {
  if (wide && i + 8 <= n) {
    float f[8];
    if constexpr (T == kF32In) {
      __builtin_memcpy(f, static_cast<const float*>(row) + i, 32);
    } else {
      const u4 v = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(row) + i);
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = sb_to_f32<T == kBF16In>(static_cast<uint16_t>(d[e >> 1] >> (16 * (e & 1))));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) key[e] = key_of(f[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) key[e] = i + e < n ? key_of(load_logit<T>(row, i + e)) : 0;
  }
}

// The same four times, all loads before their first use where every lane's are wide.
template <int T>
__device__ __forceinline__ void load_keys32(const void* row, const int (&i)[4], int n, bool wide, uint32_t (&key)[4][8]) {
  bool inside = wide;
#pragma unroll
  for (int e = 0; e < 4; ++e) inside = inside && (i[e] + 8 <= n || i[e] >= n);
  if (__all(inside)) {
    int at[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e] = i[e] + 8 <= n ? i[e] : 0;
    if (n >= 8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) load_keys8<T>(row, at[e], 0x7FFFFFFF, true, key[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) key[e][k] = i[e] + 8 <= n ? key[e][k] : 0;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) load_keys8<T>(row, i[e], n, wide, key[e]);
  }
}

// 2^z for z <= 0: whole part by the exponent, the rest, within a half, by the
// series of exp(r ln 2) to r^11 (6e-15).
__device__ __forceinline__ double exp2_neg(double z) {
  z = fmax(z, -1000.0);
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
  __device__ __forceinline__ u64 fixed(uint32_t key) const { return static_cast<u64>(__builtin_rint(weight(key) * kFix)); }
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

template <typename V>
__device__ __forceinline__ V wave_sum(V x) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), d)));
  return x;
}
// Inclusive sums over the lanes, in their order.
template <typename V>
__device__ __forceinline__ V wave_scan(V x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const V up = __shfl_up(x, d);
    if (lane >= d) x += up;
  }
  return x;
}

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int row, int size) {
  return static_cast<const char*>(a.logits) + static_cast<int64_t>(row) * a.row_stride * size;
}

struct End {
  uint32_t key;
  uint32_t ties;
};

struct Shared {
  union {
    struct {  // the list, in index order
      uint32_t key[kList];
      int id[kList];
      u64 mass[kList];
    } list;
    struct {  // bins by value
      u64 mass[kBins];
      uint32_t count[kBins];
    } bins;
  };
  u64 digit_mass[256];
  uint32_t digit_count[256];
  u64 wave_mass[kDrawWaves];
  double wave_sum[kDrawWaves];
  uint32_t wave_count[kDrawWaves], red[kDrawWaves];
  uint32_t prefix, found;
  u64 above;
  double at;
};

}  // namespace

template <int T>
__global__ __launch_bounds__(256) void sample_stats_kernel(SampleArgs a) {
  const int row = blockIdx.y, lane = threadIdx.x & 63, n = a.vocab;
  const int first = blockIdx.x * kStatTokens + threadIdx.x * 8;
  const void* x = row_of(a, row, T == kF32In ? 4 : 2);
  uint32_t key[8];
  load_keys8<T>(x, first, n, a.wide, key);
  uint32_t top = key[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) top = max(top, key[e]);
#pragma unroll
  for (int d = 1; d < 8; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if ((lane & 7) == 0 && first < n) a.cells[static_cast<int64_t>(row) * a.cell_count + first / kCell] = top;
  const Rule r = rule_of(a, row);
  if (!r.by_piece) return;
#pragma unroll
  for (int d = 8; d < 64; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  const Weigh w = weigher(top, r.t);
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += key[e] != 0 ? w.weight(key[e]) : 0.0;
  sum = wave_sum(sum);
  if (lane == 0 && first < n) a.pieces[static_cast<int64_t>(row) * a.piece_count + first / kPiece] = sum;
}

template <int T>
__global__ __launch_bounds__(kDrawThreads) void sample_draw_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.vocab;
  const void* x = row_of(a, row, T == kF32In ? 4 : 2);
  const uint32_t* cells = a.cells + static_cast<int64_t>(row) * a.cell_count;
  const double* pieces = a.pieces + static_cast<int64_t>(row) * a.piece_count;
  const Rule rule = rule_of(a, row);
  // cells and pieces of a thread: neighbours, so that threads are in index order
  const int cells_each = (a.cell_count + kDrawThreads - 1) / kDrawThreads;
  const int c0 = min(tid * cells_each, a.cell_count), c1 = min(c0 + cells_each, a.cell_count);

  uint32_t top = 0;
  for (int c = c0; c < c1; ++c) top = max(top, cells[c]);
  top = wave_max(top);
  if (lane == 0) sh.red[wave] = top;
  if (tid == 0) sh.found = 0x7FFFFFFF;
  __syncthreads();
  top = wave_max(sh.red[lane & (kDrawWaves - 1)]);
  const Weigh w = weigher(top, rule.one ? 1.0f : rule.t);

  if (rule.one) {
    for (int c = c0; c < c1; ++c)
      if (cells[c] == top) {
        atomicMin(&sh.found, static_cast<uint32_t>(c));
        break;
      }
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

  // the whole row's weight, by pieces in index order: this thread's, and that before it
  double total = 0.0, before = 0.0, mine = 0.0;
  const int pieces_each = (a.piece_count + kDrawThreads - 1) / kDrawThreads;
  const int p0 = min(tid * pieces_each, a.piece_count), p1 = min(p0 + pieces_each, a.piece_count);
  auto piece_weight = [&](int p) {
    uint32_t m = 0;
    for (int c = p * (kPiece / kCell); c < min((p + 1) * (kPiece / kCell), a.cell_count); ++c) m = max(m, cells[c]);
    return pieces[p] * w.weight(m);
  };
  if (rule.by_piece) {
    for (int p = p0; p < p1; ++p) mine += piece_weight(p);
    const double incl = wave_scan(mine, lane);
    if (lane == 63) sh.wave_sum[wave] = incl;
    __syncthreads();
    double base = 0.0;
    for (int i = 0; i < kDrawWaves; ++i) {
      if (i == wave) base = total;
      total += sh.wave_sum[i];
    }
    const double up = __shfl_up(incl, 1);
    before = base + (lane == 0 ? 0.0 : up);
    mine = base + incl;  // from here on: the sum through this thread's pieces
  }

  if (rule.open) {
    const double want = static_cast<double>(a.u[row]) * total;
    // the piece that `want` falls in; the last of them where it reaches the total
    if (tid == 0) sh.found = 0;
    __syncthreads();
    if (before <= want && mine > want) {
      double run = before;
      int p = p0;
      for (; p < p1 - 1; ++p) {
        const double next = run + piece_weight(p);
        if (next > want) break;
        run = next;
      }
      sh.found = static_cast<uint32_t>(p) + 1;
      sh.at = run;
    }
    __syncthreads();
    if (wave != 0) return;
    const bool past = sh.found == 0;
    const int p = past ? a.piece_count - 1 : static_cast<int>(sh.found) - 1, i0 = p * kPiece + lane * 8;
    uint32_t key[8];
    load_keys8<T>(x, i0, n, a.wide, key);
    double wt[8], s = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wt[e] = key[e] != 0 ? w.weight(key[e]) : 0.0;
      s += wt[e];
    }
    const double incl = (past ? 0.0 : sh.at) + wave_scan(s, lane), edge = past ? 1e300 : want;
    const u64 hit = __ballot(incl > edge), some = __ballot(s > 0.0);
    // rounding may leave the piece's own sum a hair short of its weight: its last token with weight then
    const int src = hit != 0 ? __ffsll(hit) - 1 : 63 - __clzll(some | 1);
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
      a.probs[row] = static_cast<float>(chosen / total);
    }
    return;
  }

  // exclusive place of this thread's `count` among all threads', in order
  auto place = [&](uint32_t count, uint32_t& all) {
    const uint32_t incl = wave_scan(count, lane);
    __syncthreads();
    if (lane == 63) sh.wave_count[wave] = incl;
    __syncthreads();
    uint32_t base = 0;
    all = 0;
    for (int i = 0; i < kDrawWaves; ++i) {
      if (i == wave) base = all;
      all += sh.wave_count[i];
    }
    return base + incl - count;
  };

  u64 outer_mass = 0;  // of the ties that the outer end keeps
  auto row_key = [&](int i) { return key_of(load_logit<T>(x, i)); };
  // the end of the prefix, digit by digit (8 bits), of the list's `m` tokens or the row's; by count, or by weight of
  // those up to `end`.  `above`: what is larger than all of them
  auto find_end = [&](bool listing, int m, bool by_mass, End end, double want, u64 above) {
    uint32_t prefix = 0, mask = 0;
#pragma clang loop unroll(disable)
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) {
        sh.digit_mass[tid] = 0;
        sh.digit_count[tid] = 0;
      }
      __syncthreads();
#pragma clang loop unroll(disable)
      for (int i = tid; i < m; i += kDrawThreads) {
        const uint32_t ky = listing ? sh.list.key[i] : row_key(i);
        if ((ky & mask) != prefix || ky < end.key) continue;
        const uint32_t d = (ky >> shift) & 255u;
        atomicAdd(&sh.digit_count[d], 1u);
        if (by_mass && ky > end.key) atomicAdd(&sh.digit_mass[d], listing ? sh.list.mass[i] : w.fixed(ky));
      }
      __syncthreads();
      if (wave == 0) {  // four digits a lane, the largest first
        u64 here[4], sum = 0;
        uint32_t some = 0;
        const uint32_t end_digit = (end.key & mask) == prefix && end.key != 0 ? (end.key >> shift) & 255u : 256u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t d = 255u - (lane * 4 + j);
          const uint32_t cnt = sh.digit_count[d];
          here[j] = by_mass ? sh.digit_mass[d] : cnt;
          // the ties at the outer end belong to the digit that holds it
          if (by_mass && cnt != 0 && d == end_digit) here[j] += outer_mass;
          some |= cnt != 0 ? 1u << j : 0;
          sum += here[j];
        }
        u64 run = above + wave_scan(sum, lane) - sum;
        int pick = -1, last = -1;
        u64 pick_run = 0, last_run = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((some >> j) & 1u) {
            last = j;
            last_run = run;
            if (pick < 0 && static_cast<double>(run + here[j]) >= want) {
              pick = j;
              pick_run = run;
            }
          }
          run += here[j];
        }
        const u64 hit = __ballot(pick >= 0), any = __ballot(last >= 0);
        // rounding of `want` may leave the sums short of it: the smallest that is there then
        const int src = hit != 0 ? __ffsll(hit) - 1 : 63 - __clzll(any | 1);
        if (lane == src) {
          const int j = hit != 0 ? pick : max(last, 0);
          sh.prefix = prefix | ((255u - (lane * 4 + j)) << shift);
          sh.above = hit != 0 ? pick_run : last_run;
        }
      }
      __syncthreads();
      prefix = sh.prefix;
      above = sh.above;
      mask |= 255u << shift;
    }
    End e{prefix, 1};
    const double each = by_mass ? static_cast<double>(w.fixed(prefix)) : 1.0;
    double ties = each > 0.0 ? ceil((want - static_cast<double>(above)) / each) : 1.0;
    ties = fmin(fmax(ties, 1.0), 4294967295.0);
    e.ties = static_cast<uint32_t>(ties);
    if (by_mass && prefix == end.key) e.ties = min(e.ties, end.ties);
    return e;
  };

  // bins by value: equal widths from the largest down; the last one holds all that is further
  const float top_x = value_of(top);
  auto bin_of = [&](uint32_t key, float scale) {
    const float d = (top_x - value_of(key)) * scale;
    return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
  };
  // the first bin at which `want` is reached, and what lies before it; -1: none.  Two bins a thread.
  auto reach = [&](bool by_mass, double want, u64& above, uint32_t& inside) {
    const u64 b0 = by_mass ? sh.bins.mass[2 * tid] : sh.bins.count[2 * tid];
    const u64 b1 = by_mass ? sh.bins.mass[2 * tid + 1] : sh.bins.count[2 * tid + 1];
    const u64 incl = wave_scan(b0 + b1, lane);
    if (lane == 63) sh.wave_mass[wave] = incl;
    if (tid == 0) sh.found = 0;
    __syncthreads();
    u64 base = 0;
    for (int i = 0; i < wave; ++i) base += sh.wave_mass[i];
    const u64 start = base + incl - b0 - b1;
    if (static_cast<double>(start) < want && static_cast<double>(start + b0 + b1) >= want) {
      const bool second = static_cast<double>(start + b0) < want;
      sh.found = 2 * tid + (second ? 1 : 0) + 1;
      sh.above = start + (second ? b0 : 0);
    }
    __syncthreads();
    above = sh.above;
    const int bin = static_cast<int>(sh.found) - 1;
    inside = bin >= 0 ? sh.bins.count[bin] : 0;
    __syncthreads();
    return bin;
  };
  const bool finite = top_x - top_x == 0.0f;

  // A bound that no kept token is below.
  uint32_t low = 0;
  const bool limit_k = rule.k < n;
  const int guess = limit_k ? rule.k : rule.p < 1.0f && !(rule.min_p > 0.0f) ? min(1024, a.cell_count / 2) : 0;
  if (guess > 0 && guess <= a.cell_count && guess <= kList && finite) {
    // the guess-th largest cell, to within a bin: at least that many tokens reach its smallest member
    const float scale = static_cast<float>(kBins) / fminf(fmaxf(40.0f * rule.t, 1e-30f), 1e30f);
    for (int i = tid; i < kBins; i += kDrawThreads) sh.bins.count[i] = 0;
    __syncthreads();
    for (int c = c0; c < c1; ++c) atomicAdd(&sh.bins.count[bin_of(cells[c], scale)], 1u);
    __syncthreads();
    u64 above;
    uint32_t inside;
    const int bin = reach(false, static_cast<double>(guess), above, inside);
    if (bin >= 0 && bin < kBins - 1) {
      uint32_t least = 0xFFFFFFFFu;
      for (int c = c0; c < c1; ++c)
        if (bin_of(cells[c], scale) <= bin) least = min(least, cells[c]);
      least = ~wave_max(~least);
      if (lane == 0) sh.red[wave] = least;
      __syncthreads();
      low = ~wave_max(~sh.red[lane & (kDrawWaves - 1)]);
      __syncthreads();
    }
  }
  const bool floor = rule.min_p > 0.0f;
  // top_p of the top_k needs the weight of all of those, also below min_p
  if (floor && finite && !(limit_k && rule.p < 1.0f)) {
    // w >= min_p: x >= top + t ln(min_p), with a margin for its rounding
    const double edge = w.top_value + static_cast<double>(rule.t) * log(static_cast<double>(rule.min_p));
    const double less = edge - 1e-6 * (fabs(edge) + fabs(w.top_value));
    if (less > -3e38) low = max(low, key_of(static_cast<float>(less)));
  }

  if (n <= kList) low = 1;  // the whole row is a list

  // the tokens of `from` and up, in index order, from cells that reach `from`; false where they are too many
  int listed = 0;
  auto gather_cells = [&](uint32_t from) {
    uint32_t hits = 0, all = 0;
    for (int c = c0; c < c1; ++c) hits += cells[c] >= from;
    uint32_t at = place(hits, all);
    if (all > kList) return false;
    int* hit_cells = reinterpret_cast<int*>(sh.list.mass);  // the weights come last
    for (int c = c0; c < c1; ++c)
      if (cells[c] >= from) hit_cells[at++] = c;
    __syncthreads();
    // a step of a wave: 8 cells, 8 tokens a lane
    const int steps = (static_cast<int>(all) + 7) / 8, each = (steps + kDrawWaves - 1) / kDrawWaves;
    const int h0 = min(wave * each * 8, static_cast<int>(all)), h1 = min(h0 + each * 8, static_cast<int>(all));
    // once to count, once to write
    at = 0;
    uint32_t own = 0;
#pragma clang loop unroll(disable)
    for (int round = 0; round < 2; ++round) {
#pragma clang loop unroll(disable)
      for (int j = h0; j < h1; j += 32) {
        uint32_t key[4][8];
        int first[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = j + e * 8 + (lane >> 3);
          first[e] = c < h1 ? hit_cells[c] * kCell + (lane & 7) * 8 : n;
        }
        load_keys32<T>(x, first, n, a.wide, key);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t count = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) count += key[e][i] >= from;
          if (round == 0) {
            own += count;
            continue;
          }
          const uint32_t incl = wave_scan(count, lane);
          uint32_t to = at + incl - count;
          at += __shfl(incl, 63);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (key[e][i] >= from) {
              sh.list.key[to] = key[e][i];
              sh.list.id[to] = first[e] + i;
              ++to;
            }
        }
      }
      if (round == 0) {
        own = wave_sum(own);
        at = place(lane == 0 ? own : 0, all);  // its barriers: every wave has its cells
        if (all > kList) return false;
        at = __shfl(at, 0);
      }
    }
    __syncthreads();
    for (int i = tid; i < static_cast<int>(all); i += kDrawThreads) sh.list.mass[i] = w.fixed(sh.list.key[i]);
    listed = static_cast<int>(all);
    __syncthreads();
    return true;
  };

  bool small = low != 0 && gather_cells(low);
  const double least = floor ? static_cast<double>(rule.min_p) * kFix : 0.0;  // of a kept token's integer weight
  if (small && listed <= kShort) {
    // a short list: each token's place, and the weight before it, from a look at all others
    uint32_t key = 0, rank = 0;
    u64 mass = 0, ahead = 0;
    if (tid < listed) {
      key = sh.list.key[tid];
      mass = sh.list.mass[tid];
      for (int j = 0; j < listed; ++j) {
        const uint32_t other = sh.list.key[j];
        const bool earlier = other > key || (other == key && j < tid);
        rank += earlier;
        ahead += earlier ? sh.list.mass[j] : 0;
      }
    }
    const bool within = tid < listed && rank < static_cast<uint32_t>(rule.k);
    u64 held = 0;
    if (wave < kShort / 64) held = wave_sum(within ? mass : 0);
    if (lane == 0) sh.wave_mass[wave] = held;
    __syncthreads();
    held = 0;
    for (int i = 0; i < kShort / 64; ++i) held += sh.wave_mass[i];
    const double want = static_cast<double>(rule.p) * (limit_k ? static_cast<double>(held) : total * kFix);
    // without top_k the list is a guess: it has to hold the whole prefix, or all that min_p leaves of it
    if (rule.p >= 1.0f || limit_k || floor || static_cast<double>(held) >= want) {
      const bool kept = within && (rank == 0 || ((rule.p >= 1.0f || static_cast<double>(ahead) < want) &&
                                                 static_cast<double>(mass) >= least));
      if (tid < kShort) sh.digit_mass[tid] = kept ? mass : 0;
      __syncthreads();
      if (wave != 0) return;
      constexpr int kEach = kShort / 64;
      u64 m[kEach], sum = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        m[e] = sh.digit_mass[lane * kEach + e];
        sum += m[e];
      }
      const u64 incl = wave_scan(sum, lane), all = __shfl(incl, 63);
      const double target = static_cast<double>(a.u[row]) * static_cast<double>(all);
      const u64 hit = __ballot(static_cast<double>(incl) > target), some = __ballot(sum != 0);
      // u * total may reach the total: the last token with weight then
      const int src = hit != 0 ? __ffsll(hit) - 1 : 63 - __clzll(some | 1);
      if (lane == src) {
        u64 run = incl - sum;
        int pick = -1, last = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          run += m[e];
          if (m[e] != 0) last = e;
          if (pick < 0 && hit != 0 && static_cast<double>(run) > target) pick = e;
        }
        if (pick < 0) pick = last;
        const int i = lane * kEach + pick;
        a.tokens[row] = sh.list.id[i];
        a.probs[row] = static_cast<float>(w.weight(sh.list.key[i]) * kFix / static_cast<double>(all));
      }
      return;
    }
  }
  const float fine = static_cast<float>(kBins) / fminf(fmaxf(40.0f * rule.t, 1e-30f), 1e30f);
  End end{0, 0xFFFFFFFFu};
  // by count, then by weight; a list that turns out too short leaves the second round to the row
#pragma clang loop unroll(disable)
  for (int round = 0; round < 2; ++round) {
    const bool by_mass = round != 0;
    if (by_mass ? !(rule.p < 1.0f) : !limit_k || (small && rule.k >= listed)) continue;
    double want = static_cast<double>(rule.k);
    outer_mass = by_mass && end.key != 0 ? end.ties * w.fixed(end.key) : 0;
    bool listing = small, done = false;
    if (by_mass) {
      u64 s = 0;
      if (small || limit_k) {  // the weight up to the outer end
        const int m = small ? listed : n;
#pragma clang loop unroll(disable)
        for (int i = tid; i < m; i += kDrawThreads) {
          const uint32_t key = small ? sh.list.key[i] : row_key(i);
          if (key > end.key) s += small ? sh.list.mass[i] : w.fixed(key);
        }
        s = wave_sum(s);
        __syncthreads();
        if (lane == 0) sh.wave_mass[wave] = s;
        __syncthreads();
        s = outer_mass;
        for (int i = 0; i < kDrawWaves; ++i) s += sh.wave_mass[i];
      }
      want = static_cast<double>(rule.p) * (limit_k ? static_cast<double>(s) : total * kFix);
      // without top_k the list is a guess: it has to hold the whole prefix, or all that min_p leaves of it
      if (small && !limit_k && !(static_cast<double>(s) >= want)) {
        if (floor) done = true;
        else small = listing = false;
      }
    }
    if (done) continue;
    int m = small ? listed : n;
    u64 above = 0;
    if (!small && finite) {
      // the row: the tokens of the bin in which the prefix ends become the list
      __syncthreads();
      for (int i = tid; i < kBins; i += kDrawThreads) {
        sh.bins.mass[i] = 0;
        sh.bins.count[i] = 0;
      }
      __syncthreads();
      int bin = -1;
      uint32_t inside = 0;
#pragma clang loop unroll(disable)
      for (int pass = 0; pass < 2; ++pass) {
#pragma clang loop unroll(disable)
        for (int i = tid * 8; i < n; i += kDrawThreads * 8) {
          uint32_t key[8];
          load_keys8<T>(x, i, n, a.wide, key);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int b = bin_of(key[e], fine);
            if (key[e] == 0 || key[e] < end.key || (pass == 1 && b != bin)) continue;
            const u64 mass = by_mass ? w.fixed(key[e]) : 0;
            if (pass == 0) {
              atomicAdd(&sh.bins.count[b], 1u);
              if (by_mass && key[e] > end.key) atomicAdd(&sh.bins.mass[b], mass);
            } else {  // in any order: only their keys and weights count here
              const uint32_t to = atomicAdd(&sh.found, 1u);
              sh.list.key[to] = key[e];
              sh.list.mass[to] = mass;
            }
          }
        }
        __syncthreads();
        if (pass == 0) {
          if (tid == 0 && outer_mass != 0) sh.bins.mass[bin_of(end.key, fine)] += outer_mass;
          __syncthreads();
          bin = reach(by_mass, want, above, inside);
          if (bin < 0 || inside > kList) {
            above = 0;
            break;
          }
          if (tid == 0) sh.found = 0;
          __syncthreads();
        } else {
          listing = true;
          m = static_cast<int>(sh.found);
        }
      }
    }
    end = find_end(listing, m, by_mass, end, want, above);
    __syncthreads();
  }

  // min_p: an end whose weight is below it keeps no ties, others are looked at one by one
  const u64 end_mass = end.key != 0 ? w.fixed(end.key) : 0;
  if (floor && end.key != 0 && static_cast<double>(end_mass) < least) end.ties = 0;

  // The draw, in index order: kept weight and ties wave by wave, then within
  // the wave that the border falls in.
  const int m = small ? listed : n;
  const int seg = ((m + kDrawWaves - 1) / kDrawWaves + kPiece - 1) / kPiece * kPiece;
  const int from = min(wave * seg, m), upto = min(from + seg, m);
  auto eight = [&](int at, u64 (&mass)[8], uint32_t& eq) {  // this lane's 8 of a step; eq: one bit a tie
    eq = 0;
    uint32_t key[8];
    const int i = at + lane * 8;
    if (small) {
#pragma unroll
      for (int e = 0; e < 8; ++e) key[e] = i + e < upto ? sh.list.key[i + e] : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mass[e] = i + e < upto ? sh.list.mass[i + e] : 0;
    } else {
      load_keys8<T>(x, i, upto, a.wide, key);
#pragma unroll
      for (int e = 0; e < 8; ++e) mass[e] = w.fixed(key[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (key[e] == end.key && key[e] != 0) eq |= 1u << e;
      if (key[e] <= end.key || static_cast<double>(mass[e]) < least) mass[e] = 0;
    }
  };
  auto with_ties = [&](u64 v, uint32_t eq) { return v + min(eq, end.ties) * end_mass; };
  u64 run = 0, all = 0;
  uint32_t run_eq = 0;
  double edge = 0.0;
  // once to add this wave's tokens, once, in the wave that the border falls in, to find the token
#pragma clang loop unroll(disable)
  for (int round = 0; round < 2; ++round) {
#pragma clang loop unroll(disable)
    for (int at = from; at < upto; at += kPiece) {
      u64 mass[8];
      uint32_t eq;
      eight(at, mass, eq);
      u64 own = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) own += mass[e];
      const uint32_t cnt = __popc(eq);
      if (round == 0) {
        run += own;
        run_eq += cnt;
        continue;
      }
      const u64 pre = wave_scan(own, lane);
      const uint32_t pre_eq = wave_scan(cnt, lane);
      const u64 hit = __ballot(static_cast<double>(with_ties(run + pre, run_eq + pre_eq)) > edge);
      if (hit != 0) {
        if (lane == __ffsll(hit) - 1) {
          u64 c = run + pre - own;
          uint32_t ce = run_eq + pre_eq - cnt;
          int pick = -1;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c += mass[e];
            ce += (eq >> e) & 1u;
            if (pick < 0 && static_cast<double>(with_ties(c, ce)) > edge) pick = e;
          }
          const int i = at + lane * 8 + max(pick, 0);
          a.tokens[row] = small ? sh.list.id[i] : i;
          a.probs[row] = static_cast<float>(w.weight(small ? sh.list.key[i] : row_key(i)) * kFix / static_cast<double>(all));
        }
        break;
      }
      run += __shfl(pre, 63);
      run_eq += __shfl(pre_eq, 63);
    }
    if (round == 0) {
      const u64 sum = wave_sum(run);
      const uint32_t ties = wave_sum(run_eq);
      __syncthreads();
      if (lane == 0) {
        sh.wave_mass[wave] = sum;
        sh.wave_count[wave] = ties;
      }
      __syncthreads();
      u64 mass_all = 0;
      uint32_t eq_all = 0;
      for (int i = 0; i < kDrawWaves; ++i) {
        if (i == wave) {
          run = mass_all;
          run_eq = eq_all;
        }
        mass_all += sh.wave_mass[i];
        eq_all += sh.wave_count[i];
      }
      all = with_ties(mass_all, eq_all);
      const double target = static_cast<double>(a.u[row]) * static_cast<double>(all);
      const u64 start = with_ties(run, run_eq), stop = with_ties(run + sum, run_eq + ties);
      // the wave whose tokens cross the border; the last with weight where u * total reaches the total
      const bool last = static_cast<double>(all) <= target && stop == all && start < all;
      if (!last && !(static_cast<double>(start) <= target && static_cast<double>(stop) > target)) return;
      edge = last ? static_cast<double>(all) * (1.0 - 1e-15) : target;
    }
  }
}

namespace {

template <int T>
hipError_t launch_sample_type(const SampleArgs& a) {
  for (int r0 = 0; r0 < a.rows; r0 += 65535) {  // rows of one grid
    SampleArgs b = a;
    const int rows = a.rows - r0 < 65535 ? a.rows - r0 : 65535;
    b.rows = rows;
    b.logits = static_cast<const char*>(a.logits) + static_cast<int64_t>(r0) * a.row_stride * (T == kF32In ? 4 : 2);
    b.u += r0;
    if (b.temperature) b.temperature += r0;
    if (b.top_k) b.top_k += r0;
    if (b.top_p) b.top_p += r0;
    if (b.min_p) b.min_p += r0;
    b.tokens += r0;
    b.probs += r0;
    const unsigned parts = static_cast<unsigned>((a.vocab + kStatTokens - 1) / kStatTokens);
    hipLaunchKernelGGL(sample_stats_kernel<T>, dim3(parts, static_cast<unsigned>(rows)), dim3(256), 0, a.stream, b);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_draw_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(kDrawThreads), 0, a.stream, b);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& given, const DeviceInfo& dev) {
  SampleArgs a = given;
  const int size = a.type == kF32In ? 4 : 2;
  a.wide = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && (a.rows == 1 || (a.row_stride * size) % 16 == 0);
  a.cell_count = (a.vocab + kCell - 1) / kCell;
  a.piece_count = (a.vocab + kPiece - 1) / kPiece;
  const int64_t held = a.rows < 65535 ? a.rows : 65535;
  const size_t piece_bytes = static_cast<size_t>(held) * a.piece_count * 8, cell_bytes = static_cast<size_t>(held) * a.cell_count * 4;
  return with_split_workspace(dev, a.stream, piece_bytes + cell_bytes, [&](float* ws) {
    a.pieces = reinterpret_cast<double*>(ws);
    a.cells = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(ws) + piece_bytes);
    if (a.type == kF16In) return launch_sample_type<kF16In>(a);
    if (a.type == kBF16In) return launch_sample_type<kBF16In>(a);
    return launch_sample_type<kF32In>(a);
  });
}

}  // namespace mxq
