// Drawing the next token from logits with temperature, top-k, top-p and min-p,
// given a uniform number.
//
// With w_i = exp((x_i - max x) / temperature), the kept tokens are a prefix of
// the descending order (equals by index): at most top_k of them, the shortest
// that reaches top_p of the weight of those, and w_i >= min_p.  The token drawn
// is the first, in index order, whose running sum of kept weights exceeds
// u * their total.
//
// Which token a border falls on is a whole number, so weights are taken in
// f64 and summed as integers of 2^-43: sums are then the same in any order,
// whatever threads and atomics do, and a border is off by 2^-44 a token of
// a total that is at least 1.
//
// A prefix is held as (key, ties): the value at its end, as an ordered 32-bit
// key, and how many of the tokens equal to it belong to it, the first by index.
// Its end is found digit by digit, 8 bits at a time, in histograms of counts or
// of weight.
#include "mxq_device.h"
#include "serve_internal.h"

namespace mxq {

namespace {

constexpr int kSampleThreads = 1024, kSampleWaves = 16, kPiece = 512;  // a wave's step: 8 tokens a lane
constexpr double kFix = 8796093022208.0;  // 2^43
typedef unsigned long long u64;

enum { kF16In = 0, kBF16In = 1, kF32In = 2 };

// NaN counts as -inf, -0 as 0; larger values have larger keys.
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

// Weight of a key, and its integer.
struct Weigh {
  uint32_t top;
  double top_value, t;
  __device__ __forceinline__ double weight(uint32_t key) const {
    return key == top ? 1.0 : exp((static_cast<double>(value_of(key)) - top_value) / t);
  }
  __device__ __forceinline__ u64 fixed(uint32_t key) const { return static_cast<u64>(__builtin_rint(weight(key) * kFix)); }
};

__device__ __forceinline__ u64 wave_sum(u64 x) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d);
  return x;
}

struct End {
  uint32_t key;
  uint32_t ties;
};

struct Shared {
  u64 mass[256];
  uint32_t count[256];
  u64 wave_mass[kSampleWaves];
  uint32_t wave_eq[kSampleWaves], red[kSampleWaves];
  uint32_t prefix, ties;
  u64 above;
  int token, wave;
  double prob;
};

}  // namespace

template <int T>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.vocab;
  const void* x = static_cast<const char*>(a.logits) + static_cast<int64_t>(row) * a.row_stride * (T == kF32In ? 4 : 2);
  const float temp = a.temperature ? a.temperature[row] : a.temperature_all;
  int k = a.top_k ? a.top_k[row] : a.top_k_all;
  float p = a.top_p ? a.top_p[row] : a.top_p_all;
  const float min_p = a.min_p ? a.min_p[row] : a.min_p_all;
  const bool one = !(temp > 0.0f) || !(p > 0.0f) || !(min_p <= 1.0f) || k == 1;  // the largest, the first of equals
  if (k <= 0 || k > n) k = n;

  // the largest
  uint32_t top = 0;
  for (int i = tid; i < n; i += kSampleThreads) top = max(top, key_of(load_logit<T>(x, i)));
#pragma unroll
  for (int d = 32; d > 0; d /= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if (lane == 0) sh.red[wave] = top;
  __syncthreads();
  top = sh.red[lane & 15];
#pragma unroll
  for (int d = 8; d > 0; d /= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  const Weigh w{top, static_cast<double>(value_of(top)), one ? 1.0 : static_cast<double>(temp)};

  // the end of the prefix among tokens up to `end`: by count, or by weight
  auto find_end = [&](bool by_mass, End end, double want) {
    constexpr int rounds = T == kBF16In ? 2 : T == kF16In ? 3 : 4;  // the other digits are the same for all
    uint32_t prefix = 0, mask = 0;
    u64 above = 0;
    for (int r = 0; r < rounds; ++r) {
      const int shift = 24 - 8 * r;
      if (tid < 256) {
        sh.mass[tid] = 0;
        sh.count[tid] = 0;
      }
      __syncthreads();
      for (int i = tid; i < n; i += kSampleThreads) {
        const uint32_t key = key_of(load_logit<T>(x, i));
        if ((key & mask) != prefix || key < end.key) continue;
        const uint32_t d = (key >> shift) & 255u;
        atomicAdd(&sh.count[d], 1u);
        if (by_mass && key > end.key) atomicAdd(&sh.mass[d], w.fixed(key));
      }
      __syncthreads();
      if (tid == 0) {
        u64 cum = above;
        int d = 255;
        for (; d >= 0; --d) {
          const uint32_t low = prefix | (static_cast<uint32_t>(d) << shift);
          u64 here = by_mass ? sh.mass[d] : sh.count[d];
          // the ties at the outer end belong to the digit that holds it
          if (by_mass && end.key != 0 && sh.count[d] != 0 && (end.key & (mask | (255u << shift))) == low) here += end.ties * w.fixed(end.key);
          if (sh.count[d] != 0 && static_cast<double>(cum + here) >= want) break;
          cum += here;
        }
        if (d < 0) d = static_cast<int>((end.key >> shift) & 255u);
        sh.prefix = prefix | (static_cast<uint32_t>(d) << shift);
        sh.above = cum;
      }
      __syncthreads();
      prefix = sh.prefix;
      above = sh.above;
      mask |= 255u << shift;
    }
    // digits that no round looked at: ones for negative values, zeros for others
    End e;
    e.key = prefix & 0x80000000u ? prefix : prefix | ~mask;
    const double each = by_mass ? static_cast<double>(w.fixed(e.key)) : 1.0;
    double ties = each > 0.0 ? ceil((want - static_cast<double>(above)) / each) : 1.0;
    ties = fmin(fmax(ties, 1.0), 4294967295.0);
    e.ties = static_cast<uint32_t>(ties);
    if (by_mass && e.key == end.key) e.ties = min(e.ties, end.ties);
    return e;
  };

  End end{0, 0xFFFFFFFFu};
  if (one) {
    end = End{top, 1};
  } else {
    if (k < n) end = find_end(false, End{0, 0xFFFFFFFFu}, static_cast<double>(k));
    if (p < 1.0f) {
      // the weight of the top_k
      u64 sum = 0;
      for (int i = tid; i < n; i += kSampleThreads) {
        const uint32_t key = key_of(load_logit<T>(x, i));
        if (key > end.key) sum += w.fixed(key);
      }
      sum = wave_sum(sum);
      if (lane == 0) sh.wave_mass[wave] = sum;
      __syncthreads();
      sum = 0;
      for (int i = 0; i < kSampleWaves; ++i) sum += sh.wave_mass[i];
      if (k < n) sum += end.ties * w.fixed(end.key);
      __syncthreads();
      end = find_end(true, end, static_cast<double>(p) * static_cast<double>(sum));
    }
  }
  // min_p: an end whose weight is below it keeps no ties, others are looked at one by one
  const bool floor = min_p > 0.0f && !one;
  if (floor && end.key != 0 && w.weight(end.key) < static_cast<double>(min_p)) end.ties = 0;
  const u64 end_mass = end.key != 0 ? w.fixed(end.key) : 0;

  // kept weight and ties, wave by wave in index order
  const int seg = ((n + kSampleWaves - 1) / kSampleWaves + kPiece - 1) / kPiece * kPiece;
  const int from = min(wave * seg, n), upto = min(from + seg, n);
  auto piece = [&](int at, u64 (&mass)[8], uint32_t& eq) {  // this lane's 8 tokens from `at` on; eq: one bit a tie
    eq = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = at + lane * 8 + e;
      mass[e] = 0;
      if (i >= upto) continue;
      const uint32_t key = key_of(load_logit<T>(x, i));
      if (key > end.key) {
        const double v = w.weight(key);
        if (!floor || v >= static_cast<double>(min_p)) mass[e] = static_cast<u64>(__builtin_rint(v * kFix));
      } else if (key == end.key) {
        eq |= 1u << e;
      }
    }
  };
  u64 sum = 0;
  uint32_t ties = 0;
  for (int at = from; at < upto; at += kPiece) {
    u64 mass[8];
    uint32_t eq;
    piece(at, mass, eq);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += mass[e];
    ties += __popc(eq);
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) ties += __shfl_xor(static_cast<int>(ties), d);
  if (lane == 0) {
    sh.wave_mass[wave] = sum;
    sh.wave_eq[wave] = ties;
  }
  if (tid == 0) sh.token = -1;
  __syncthreads();
  u64 before = 0, total = 0;
  uint32_t eq_before = 0, eq_total = 0;
  for (int i = 0; i < kSampleWaves; ++i) {
    if (i < wave) {
      before += sh.wave_mass[i];
      eq_before += sh.wave_eq[i];
    }
    total += sh.wave_mass[i];
    eq_total += sh.wave_eq[i];
  }
  auto with_ties = [&](u64 m, uint32_t eq) { return m + min(eq, end.ties) * end_mass; };
  const u64 all = with_ties(total, eq_total);
  const double want = static_cast<double>(a.u[row]) * static_cast<double>(all);
  const u64 low = with_ties(before, eq_before), high = with_ties(before + sum, eq_before + ties);
  // the wave whose tokens cross the border; the last with weight where u * total reaches the total
  const bool last = static_cast<double>(all) <= want && high == all && low < all;
  if ((static_cast<double>(low) <= want && static_cast<double>(high) > want) || last) {
    const double edge = last ? static_cast<double>(all) * (1.0 - 1e-15) : want;
    u64 run = before;
    uint32_t run_eq = eq_before;
    for (int at = from; at < upto; at += kPiece) {
      u64 mass[8];
      uint32_t eq;
      piece(at, mass, eq);
      u64 mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine += mass[e];
      uint32_t cnt = __popc(eq);
      u64 pre = mine;
      uint32_t pre_eq = cnt;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const u64 up = __shfl_up(pre, d);
        const uint32_t up_eq = __shfl_up(static_cast<int>(pre_eq), d);
        if (lane >= d) {
          pre += up;
          pre_eq += up_eq;
        }
      }
      const u64 hit = __ballot(static_cast<double>(with_ties(run + pre, run_eq + pre_eq)) > edge);
      if (hit != 0) {
        if (lane == __ffsll(hit) - 1) {
          u64 c = run + pre - mine;
          uint32_t ce = run_eq + pre_eq - cnt;
          bool done = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c += mass[e];
            ce += (eq >> e) & 1u;
            if (!done && static_cast<double>(with_ties(c, ce)) > edge) {
              done = true;
              const int i = at + lane * 8 + e;
              a.tokens[row] = i;
              a.probs[row] = static_cast<float>(w.weight(key_of(load_logit<T>(x, i))) * kFix / static_cast<double>(all));
            }
          }
        }
        break;
      }
      run += __shfl(pre, 63);
      run_eq += __shfl(static_cast<int>(pre_eq), 63);
    }
  }
}

hipError_t launch_sample(const SampleArgs& a) {
  const dim3 grid(static_cast<unsigned>(a.rows)), block(kSampleThreads);
  if (a.type == kF16In) hipLaunchKernelGGL(sample_kernel<kF16In>, grid, block, 0, a.stream, a);
  else if (a.type == kBF16In) hipLaunchKernelGGL(sample_kernel<kBF16In>, grid, block, 0, a.stream, a);
  else hipLaunchKernelGGL(sample_kernel<kF32In>, grid, block, 0, a.stream, a);
  return hipGetLastError();
}

}  // namespace mxq
