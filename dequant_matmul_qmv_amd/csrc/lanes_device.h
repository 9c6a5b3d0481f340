// Sums, scans and largest values over a wave's 64 lanes by DPP moves.  Whole
// waves: every lane takes part.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace mxq {

typedef unsigned long long u64;

// x of another lane by a DPP control, 0 where there is none (or the lane's row
// of 16 is not in `rows`): a few cycles, where a shuffle through LDS takes 100.
template <int CTRL, int ROWS, typename V>
__device__ __forceinline__ V lane_move(V x) {
  static_assert(sizeof(V) == 4 || sizeof(V) == 8, "one or two registers");
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false));
  } else {
    const u64 w = __builtin_bit_cast(u64, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(w >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(V, (static_cast<u64>(hi) << 32) | lo);
  }
}
template <typename V>
__device__ __forceinline__ V last_lane(V x) {
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
  } else {
    const u64 w = __builtin_bit_cast(u64, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(w), 63), hi = __builtin_amdgcn_readlane(static_cast<int>(w >> 32), 63);
    return __builtin_bit_cast(V, (static_cast<u64>(hi) << 32) | lo);
  }
}
// Inclusive sums over the lanes, in their order: within rows of 16, then the
// rows' last lanes handed on.
template <typename V>
__device__ __forceinline__ V wave_scan(V x) {
  x += lane_move<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8
  x += lane_move<0x112, 0xF>(x);
  x += lane_move<0x114, 0xF>(x);
  x += lane_move<0x118, 0xF>(x);
  x += lane_move<0x142, 0xA>(x);  // row_bcast 15, 31
  x += lane_move<0x143, 0xC>(x);
  return x;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V x) { return last_lane(wave_scan(x)); }
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, lane_move<0x111, 0xF>(x));
  x = max(x, lane_move<0x112, 0xF>(x));
  x = max(x, lane_move<0x114, 0xF>(x));
  x = max(x, lane_move<0x118, 0xF>(x));
  x = max(x, lane_move<0x142, 0xA>(x));
  x = max(x, lane_move<0x143, 0xC>(x));
  return last_lane(x);
}
__device__ __forceinline__ u64 wave_or(u64 x) {
  x |= lane_move<0x111, 0xF>(x);
  x |= lane_move<0x112, 0xF>(x);
  x |= lane_move<0x114, 0xF>(x);
  x |= lane_move<0x118, 0xF>(x);
  x |= lane_move<0x142, 0xA>(x);
  x |= lane_move<0x143, 0xC>(x);
  return last_lane(x);
}
// How many of the lanes below this one are in `who`.
__device__ __forceinline__ int lanes_below(u64 who) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(who >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(who), 0));
}

}  // namespace mxq
