// How attention's work is divided, for both forms of the cache: parts of a few
// rows' keys, tiles of many rows, the plan of a call, and the kernels that join
// partial results.
#pragma once

#include <climits>

#include "attend_device.h"

namespace mxq {

namespace {

constexpr int kFewWaves = 4;    // of a workgroup; twice that where it takes all keys
constexpr int kChunk = 64;      // keys a wave takes at a time
constexpr int kMinChunks = 4;   // at least one chunk for each wave of a workgroup
// Tables of up to this many keys are not split: a workgroup of eight waves takes
// all keys of its rows, in two rounds at most.  8 kv heads, split and joined / not
// split, in us, a call among others and inside a graph (which then has no
// workspace to allocate):
//   1 sequence    64 values, 512 keys 11.3 / 8.8, 20.1 / 6.8; 1024 keys 11.3 / 8.8, 20.7 / 9.2
//                128 values, 512 keys 11.2 / 8.7, 19.5 / 8.8; 1024 keys 11.2 / 12.0, 18.7 / 12.4
//   32 sequences  64 values, 1024 keys 14.6 / 9.9, 23.0 / 10.5
//                128 values, 1024 keys 22.9 / 16.0, 31.1 / 16.8
// So 128 values, more than 512 keys and few sequences lose 1 us outside a graph
// and win 6 inside one; all others win both ways.
constexpr int kLoneKeys = 1024;
constexpr int kManyRows = 128;  // of a many-row tile

// One sequence's share of the few-row work.
struct Share {
  int c0, chunks;  // first 64-key chunk, and how many
  int groups;      // groups of 16 * MT rows
};
template <int MT, typename Args>
__device__ __forceinline__ Share share_of(const Args& a, int s) {
  Share r{};
  if (s >= a.seqs) return r;
  const SeqSpan q = seq_span(a, s);
  const int64_t rows = static_cast<int64_t>(q.n) * a.group;
  if (rows > a.few_rows) return r;
  r.groups = static_cast<int>((rows + 16 * MT - 1) / (16 * MT));
  const int hi = min(q.len, a.width * a.pool.block);
  const int lo = first_seen(a, q.len - q.n);
  r.c0 = lo / kChunk;
  r.chunks = max(0, hi / kChunk + (hi % kChunk != 0) - r.c0);  // (hi may be near 2^31)
  return r;
}

struct Part {
  bool any;
  int seq, base, nth;   // base: the sequence's first slot; nth: the slot within it
  int step, splits;     // chunks of a part, parts of the sequence
  Share share;
};

// Chunks of a part, of all sequences' `total`.
template <typename Args>
__device__ __forceinline__ int part_step(const Args& a, long long total) {
  // As many workgroups a compute unit as the kernel asks for, or half of them where
  // they would have its long parts; parts of whole rounds of the four waves (8 bits, 64
  // sequences: 48 us with parts of 9 chunks, 45 with 12).
  long long even = (total + a.target - 1) / a.target;
  if (even >= a.long_chunks) even *= 2;
  return static_cast<int>((max(even, static_cast<long long>(a.min_chunks)) + kFewWaves - 1) / kFewWaves * kFewWaves);
}

// Where slot `slot` lies, or (slot < 0) sequence `seq`.  Run by whole waves.
template <int MT, typename Args>
__device__ Part find_part(const Args& a, int slot, int seq) {
  const int lane = threadIdx.x & 63, hk = a.pool.kv_heads;
  long long total = 0;
  Share mine{};
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    mine = share_of<MT>(a, s0 + lane);
    total += static_cast<long long>(mine.chunks) * mine.groups * hk;
  }
  Part p{};
  p.step = part_step(a, wave_sum(total));
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    if (a.seqs > 64) mine = share_of<MT>(a, s0 + lane);
    const int splits = max(1, (mine.chunks + p.step - 1) / p.step);
    const int count = mine.groups * splits * hk;
    const int sum = wave_scan(count);
    const unsigned long long hit = slot >= 0 ? __ballot(before + sum > slot) : (seq < s0 + 64 ? 1ull << (seq - s0) : 0);
    if (hit != 0) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      p.any = true;
      p.seq = s0 + src;
      p.base = before + __builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(count, src);
      p.nth = slot - p.base;
      p.splits = __builtin_amdgcn_readlane(splits, src);
      p.share.c0 = __builtin_amdgcn_readlane(mine.c0, src);
      p.share.chunks = __builtin_amdgcn_readlane(mine.chunks, src);
      p.share.groups = __builtin_amdgcn_readlane(mine.groups, src);
      return p;
    }
    before += last_lane(sum);
  }
  return p;
}

// Whether long parts go first.  The search for them reads lens again for each of three kinds
// where there are more sequences than two registers hold: that costs more than it gives
// unless sequences may be long.  Heads of 128 over 4 bits, in us, long first / by sequence:
//   up to 8192 keys   129 sequences 60 / 67, 192 84 / 95, 256 122 / 133, 512 263 / 249
//   up to 2048 keys   256 sequences 71 / 61, 1024 538 / 325
constexpr int kKeptSeqs = 128;
template <typename Args>
__device__ __forceinline__ bool long_first_pays(const Args& a) {
  return a.seqs <= kKeptSeqs || 24 * static_cast<int64_t>(a.seqs) <= static_cast<int64_t>(a.width) * a.pool.block;
}

// The part that workgroup `index` takes where long parts go first: whole ones, then the
// sequences' ends of at least half a part, then the others.  What is left for the last
// workgroups is short (96 sequences of 5 .. 8192 keys over 4 bits: 44 us, by sequence 49,
// with two kinds instead of three 51).  Its slot is base + nth, as above.
template <int MT, typename Args>
__device__ Part find_part_long_first(const Args& a, int index) {
  const int lane = threadIdx.x & 63, hk = a.pool.kv_heads;
  long long total = 0;
  int groups = 0;
  Share last{};
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    last = share_of<MT>(a, s0 + lane);
    total += static_cast<long long>(last.chunks) * last.groups * hk;
    groups |= last.groups;
  }
  Part p{};
  // (a call of prompts alone: 4.8 us for its workgroups to find that, 7.6 by way of the kinds)
  if (!__any(groups != 0)) return p;
  p.step = part_step(a, wave_sum(total));
  const bool kept = a.seqs <= kKeptSeqs;  // in registers: `first` and `last`
  const Share first = a.seqs > 64 && kept ? share_of<MT>(a, lane) : last;
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    int before = 0, slots = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64) {
      const Share mine = kept ? (s0 == 0 ? first : last) : share_of<MT>(a, s0 + lane);
      const int rows = mine.groups * hk, whole = mine.chunks / p.step, rest = mine.chunks - whole * p.step;
      const int splits = max(1, whole + (rest > 0)), end = rest >= p.step / 2 ? 1 : 2;
      const int count = rows * (kind == 0 ? whole : kind == end ? splits - whole : 0), all = rows * splits;
      const int sum = wave_scan(count), all_sum = wave_scan(all);
      const unsigned long long hit = __ballot(before + sum > index);
      if (hit != 0) {
        const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
        p.any = true;
        p.seq = s0 + src;
        p.base = slots + __builtin_amdgcn_readlane(all_sum, src) - __builtin_amdgcn_readlane(all, src);
        p.nth = index - before - (__builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(count, src)) +
                (kind > 0 ? __builtin_amdgcn_readlane(rows * whole, src) : 0);
        p.splits = __builtin_amdgcn_readlane(splits, src);
        p.share.c0 = __builtin_amdgcn_readlane(mine.c0, src);
        p.share.chunks = __builtin_amdgcn_readlane(mine.chunks, src);
        p.share.groups = __builtin_amdgcn_readlane(mine.groups, src);
        return p;
      }
      before += last_lane(sum);
      slots += last_lane(all_sum);
    }
    index -= before;
  }
  return p;
}

// Rows a sequence gives to this kernel, in tiles.
template <typename Args>
__device__ __forceinline__ int tiles_of(const Args& a, int s) {
  if (s >= a.seqs) return 0;
  const SeqSpan q = seq_span(a, s);
  const int64_t rows = static_cast<int64_t>(q.n) * a.group;
  return rows > a.few_rows ? static_cast<int>((rows + kManyRows - 1) / kManyRows) : 0;
}

// (sequence, tile within it) of tile `index`, or with index < 0 the first tile
// of sequence `seq` in `first`.  Whole waves.
template <typename Args>
__device__ bool find_tile(const Args& a, int index, int& seq, int& first) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const int count = tiles_of(a, s0 + lane);
    const int sum = wave_scan(count);
    const unsigned long long hit = index >= 0 ? __ballot(before + sum > index) : (seq < s0 + 64 ? 1ull << (seq - s0) : 0);
    if (hit != 0) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      seq = s0 + src;
      first = before + __builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(count, src);
      return true;
    }
    before += last_lane(sum);
  }
  return false;
}

// The tiles of a call at most, and the bytes of their partial results.
template <typename Args>
int64_t many_tiles(const Args& a) {
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.group;
  // every sequence of this kernel has more than few_rows rows, and at most one partial tile
  const int64_t seqs = a.few_rows < 1 ? a.seqs : rows / a.few_rows;
  return rows / kManyRows + (seqs < a.seqs ? seqs : a.seqs);
}

template <typename Args>
size_t many_part_bytes(const Args& a) {
  return a.many_splits == 1 ? 0 : static_cast<size_t>(many_tiles(a)) * a.pool.kv_heads * a.many_splits * kManyRows * (a.pool.dim + 2) * 4;
}

}  // namespace

// One workgroup for each (token, query head): the parts of its row, 4 values a
// lane, the parts dealt over the workgroup's groups of DIM / 4 lanes.
template <int DIM, int MT, bool BF16, int THREADS, typename Args>
__global__ __launch_bounds__(THREADS) void attend_join_kernel(Args a) {
  constexpr int kLanes = DIM / 4, kTeams = THREADS / kLanes, kRows = 16 * MT;
  __shared__ float sums[kTeams][DIM];
  __shared__ float team_m[kTeams], team_l[kTeams];
  // one token a sequence, or up to `join_new`
  const int hq = blockIdx.y, seq = blockIdx.x / a.join_new, nth = blockIdx.x - seq * a.join_new;
  const SeqSpan sp = seq_span(a, seq);
  if (nth >= sp.n || static_cast<int64_t>(sp.n) * a.group > a.few_rows) return;
  const int tok = sp.t0 + nth;
  const Part part = find_part<MT>(a, -1, seq);
  if (part.splits == 1) return;
  const int hk = a.pool.kv_heads, head = hq / a.group;
  const int i = (tok - sp.t0) * a.group + hq - head * a.group, rg = i / kRows, row = i - rg * kRows;
  const int team = threadIdx.x / kLanes, d = (threadIdx.x - team * kLanes) * 4;
  float top = kNegInf, total = 0.0f;
  f4 y = f4{0, 0, 0, 0};
  // four parts at a time, so that their loads run together
  for (int s0 = team; s0 < part.splits; s0 += 4 * kTeams) {
    float2 ml[4];
    f4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = min(s0 + i * kTeams, part.splits - 1);
      // (starts that descend may give more than there are: not read)
      const int64_t slot = min(part.base + (static_cast<int64_t>(s) * part.share.groups + rg) * hk + head, static_cast<int64_t>(a.slots) - 1);
      const int64_t at = slot * kRows + row;
      ml[i] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
      v[i] = *reinterpret_cast<const f4*>(a.part + at * DIM + d);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s0 + i * kTeams >= part.splits) continue;
      const float now = fmaxf(top, ml[i].x), ref = now == kNegInf ? 0.0f : now;
      const float e0 = __builtin_amdgcn_exp2f(top - ref), w = ml[i].y * kJoinUnit * __builtin_amdgcn_exp2f(ml[i].x - ref);
      y = y * e0 + v[i] * w;
      total = total * e0 + w;
      top = now;
    }
  }
  *reinterpret_cast<f4*>(&sums[team][d]) = y;
  if (d == 0) {
    team_m[team] = top;
    team_l[team] = total;
  }
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  top = team_m[0];
#pragma unroll
  for (int t = 1; t < kTeams; ++t) top = fmaxf(top, team_m[t]);
  const float ref = top == kNegInf ? 0.0f : top;
  y = f4{0, 0, 0, 0};
  total = 0.0f;
#pragma unroll
  for (int t = 0; t < kTeams; ++t) {
    const float e = __builtin_amdgcn_exp2f(team_m[t] - ref);
    y += *reinterpret_cast<const f4*>(&sums[t][d]) * e;
    total += team_l[t] * e;
  }
  const int64_t at = static_cast<int64_t>(tok) * a.heads + hq;
  const float inv = over(total);
  uint16_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(y[e] * inv);
  *reinterpret_cast<uint2*>(a.out + at * DIM + d) = uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                                                          static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
  if (a.lse && d == 0) a.lse[at] = log_sum(ref, total / kJoinUnit);
}

// Joins a row's parts where the key axis was split: a workgroup for each token
// and as many query heads as it has groups of DIM / 4 lanes, one of them a group.
// Eight parts are read at a time (24 parts of 51 tokens over 6204 keys, the
// whole call: 33 us one by one; two parts of 1281 tokens of 16 heads: 16 us with
// a workgroup a row).
template <int DIM, bool BF16, typename Args>
__global__ __launch_bounds__(256) void attend_many_join_kernel(Args a) {
  constexpr int kLanes = DIM / 4, kTeams = 256 / kLanes;
  const int tok = blockIdx.x, hk = a.pool.kv_heads;
  int lo = 0, hi = a.seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.starts[mid] <= tok) lo = mid; else hi = mid;
  }
  int seq = lo, first = 0;
  const SeqSpan sp = seq_span(a, seq);
  if (tok < sp.t0 || tok >= sp.t0 + sp.n || static_cast<int64_t>(sp.n) * a.group <= a.few_rows) return;
  find_tile(a, -1, seq, first);
  const int team = threadIdx.x / kLanes, d = (threadIdx.x - team * kLanes) * 4, hq = blockIdx.y * kTeams + team;
  if (hq >= a.heads) return;
  const int head = hq / a.group, i = (tok - sp.t0) * a.group + hq - head * a.group;
  const int64_t tile = first + i / kManyRows;
  float top = kNegInf, total = 0.0f;
  f4 y = f4{0, 0, 0, 0};
  for (int s0 = 0; s0 < a.many_splits; s0 += 8) {
    float2 ml[8];
    f4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int s = min(s0 + e, a.many_splits - 1);
      const int64_t at = min((tile * a.many_splits + s) * hk + head, static_cast<int64_t>(a.many_units) - 1) * kManyRows + i % kManyRows;
      ml[e] = *reinterpret_cast<const float2*>(a.many_ml + at * 2);
      v[e] = *reinterpret_cast<const f4*>(a.many_part + at * DIM + d);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (s0 + e >= a.many_splits) continue;
      const float now = fmaxf(top, ml[e].x), ref = now == kNegInf ? 0.0f : now;
      const float e0 = __builtin_amdgcn_exp2f(top - ref), w = ml[e].y * kJoinUnit * __builtin_amdgcn_exp2f(ml[e].x - ref);
      y = y * e0 + v[e] * w;
      total = total * e0 + w;
      top = now;
    }
  }
  const int64_t at = static_cast<int64_t>(tok) * a.heads + hq;
  const float inv = over(total);
  uint16_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = f32_to_act_bits<BF16>(y[e] * inv);
  *reinterpret_cast<uint2*>(a.out + at * DIM + d) = uint2{static_cast<uint32_t>(o[0]) | (static_cast<uint32_t>(o[1]) << 16),
                                                          static_cast<uint32_t>(o[2]) | (static_cast<uint32_t>(o[3]) << 16)};
  if (a.lse && d == 0) a.lse[at] = log_sum(top == kNegInf ? 0.0f : top, total / kJoinUnit);
}

namespace {

// Waves of a workgroup: twice as many where it takes all keys of more than a
// round (32 rows of 128 values do not fit the registers of that many waves).
constexpr int lone_waves(int values) { return values >= 256 ? kFewWaves : 2 * kFewWaves; }
template <typename Args>
int few_waves(const Args& a, int values, bool joined) {
  return !joined && static_cast<int64_t>(a.width) * a.pool.block > kFewWaves * kChunk ? lone_waves(values) : kFewWaves;
}
// One wave a row joins where the sequences are too many to have many parts each
// (64 sequences: 45.4 -> 44.1 us).
template <typename Args>
int join_threads(const Args& a) { return 8 * static_cast<int64_t>(a.seqs) * a.pool.kv_heads >= a.target ? 64 : 256; }

template <int DIM, int MT, typename Parts, typename Args>
hipError_t launch_mt(const Args& a, unsigned slots, bool joined) {
  hipError_t e = few_waves(a, MT * DIM, joined) == kFewWaves ? Parts::template launch<DIM, MT, kFewWaves>(a, slots)
                                                             : Parts::template launch<DIM, MT, lone_waves(MT * DIM)>(a, slots);
  if (e != hipSuccess || !joined) return e;
  const dim3 grid(static_cast<unsigned>(a.seqs) * static_cast<unsigned>(a.join_new), static_cast<unsigned>(a.heads));
  if (join_threads(a) == 64) {
    if (a.bf16) hipLaunchKernelGGL((attend_join_kernel<DIM, MT, true, 64>), grid, dim3(64), 0, a.stream, a);
    else hipLaunchKernelGGL((attend_join_kernel<DIM, MT, false, 64>), grid, dim3(64), 0, a.stream, a);
  } else {
    if (a.bf16) hipLaunchKernelGGL((attend_join_kernel<DIM, MT, true, 256>), grid, dim3(256), 0, a.stream, a);
    else hipLaunchKernelGGL((attend_join_kernel<DIM, MT, false, 256>), grid, dim3(256), 0, a.stream, a);
  }
  return hipGetLastError();
}

template <typename Parts, typename Args>
hipError_t launch_few(const Args& a, int mt, unsigned slots, bool joined) {
  if (slots == 0) return hipSuccess;
  if (a.pool.dim == 64) return mt == 1 ? launch_mt<64, 1, Parts>(a, slots, joined) : launch_mt<64, 2, Parts>(a, slots, joined);
  return mt == 1 ? launch_mt<128, 1, Parts>(a, slots, joined) : launch_mt<128, 2, Parts>(a, slots, joined);
}

// Sequences of up to this many rows take the few-row kernel.
constexpr int kFewRows = 64;

// Plans a call, and launches its few-row kernel (Parts::launch) and its many-row one.
template <typename Parts, typename Args>
hipError_t launch_attend_parts(const Args& given, const DeviceInfo& dev) {
  Args a = given;
  if (a.pool.blocks == 0) a.width = 0;  // no page exists: every row is empty
  const int64_t all_rows = static_cast<int64_t>(a.tokens) * a.group, hk = a.pool.kv_heads;
  // How many new tokens a sequence has is known on the GPU alone.  One kernel
  // runs where that cannot matter; else both, each with its own sequences.
  const bool few = a.starts == nullptr || a.seqs > 1 || all_rows <= kFewRows;
  const bool many = a.starts != nullptr && all_rows > kFewRows;
  a.few_rows = !many ? INT_MAX : few ? kFewRows : 0;
  a.target = dev.num_cu * Parts::kPerUnit;
  a.long_chunks = Parts::kLongChunks;
  // the most new tokens of a sequence that the few-row kernel takes
  a.join_new = a.starts == nullptr ? 1 : many ? (kFewRows / a.group > 0 ? kFewRows / a.group : 1) : a.tokens;

  const int64_t most = a.starts == nullptr ? a.group : all_rows < kFewRows ? all_rows : kFewRows;
  const int mt = most <= 16 ? 1 : 2;
  // slots: at most `target` full parts, and one more for each (sequence, group of rows, kv head)
  int64_t few_total = all_rows;
  if (many && few_total > static_cast<int64_t>(a.seqs) * kFewRows) few_total = static_cast<int64_t>(a.seqs) * kFewRows;
  const int64_t per = 16 * mt, ends = few ? (few_total / per + a.seqs) * hk : 0;
  const bool joined = few && static_cast<int64_t>(a.width) * a.pool.block > kLoneKeys;
  a.min_chunks = joined ? kMinChunks : kLoneKeys / kChunk;
  const int64_t slots = ends + (joined ? a.target : 0);
  if (few && (!grid_fits(slots, 64 * few_waves(a, mt * a.pool.dim, joined)) ||
              (joined && !grid_fits(static_cast<int64_t>(a.seqs) * a.join_new, join_threads(a)))))
    return kTooLarge;
  a.slots = static_cast<int>(slots);
  const size_t sums = joined ? static_cast<size_t>(slots) * per * a.pool.dim * 4 : 0;
  const size_t few_bytes = joined ? sums + static_cast<size_t>(slots) * per * 8 : 0;

  // the many-row kernel's key axis is split while its tiles leave compute units idle
  a.many_splits = 1;
  if (many) {
    const int64_t tiles = many_tiles(a) * hk, stages = (static_cast<int64_t>(a.width) * a.pool.block + kChunk - 1) / kChunk;
    int64_t splits = tiles > 0 ? 2 * dev.num_cu / tiles : 1;
    if (splits > stages / 4) splits = stages / 4;
    if (splits > 32) splits = 32;
    if (splits > 1) a.many_splits = static_cast<int>(splits);
  }
  if (many && (!grid_fits(many_tiles(a) * hk * a.many_splits, 256) || (a.many_splits > 1 && !grid_fits(a.tokens, 256)))) return kTooLarge;
  const size_t many_bytes = many ? many_part_bytes(a) : 0;

  const auto enqueue = [&](float* ws) {
    a.part = ws;
    a.part_ml = ws + sums / 4;
    hipError_t e = many ? launch_many(a, ws + few_bytes / 4) : hipSuccess;
    if (e == hipSuccess && few) e = launch_few<Parts>(a, mt, static_cast<unsigned>(slots), joined);
    return e;
  };
  if (few_bytes + many_bytes == 0) return enqueue(nullptr);
  return with_split_workspace(dev, a.stream, few_bytes + many_bytes, enqueue);
}

}  // namespace

}  // namespace mxq
