// Host-side internals of the serving operators between the projections
// (rotary positions, the 8-bit paged cache, attention over it, sampling).
#pragma once

#include <string>

#include "../../include/mxq.h"
#include "mxq_internal.h"

namespace mxq {

// The calling thread's error text (api.cpp): cleared at the start of a call,
// set where a call fails.
void clear_error();
mxq_status report(mxq_status s, const std::string& msg);
mxq_status report_hip(const char* who, hipError_t e);

// q and k views: [tokens, heads, dim] with element strides for tokens and
// heads, the last dimension contiguous.  Null with 0 heads: absent.
struct RopeSide {
  const uint16_t* in;
  uint16_t* out;
  int64_t in_token, in_head, out_token, out_head;
  int heads;
};
struct RopeArgs {
  RopeSide side[2];  // q, k
  const float* inv_freq;
  const int32_t* positions;
  int64_t tokens;
  int dim, rot;
  bool interleaved, bf16;
  hipStream_t stream;
};
hipError_t launch_rope(const RopeArgs& a);

// The paged cache: k codes [blocks, kv_heads, block, dim], v codes [blocks,
// kv_heads, dim, block], scales [blocks, kv_heads].
struct KvPool {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t blocks;
  int kv_heads, block, dim;
};
struct KvAppendArgs {
  KvPool pool;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_token, k_head, v_token, v_head;
  const int32_t* table;
  int64_t table_stride;
  int width;
  const int32_t* lens;
  const int32_t* starts;  // null: one token for each sequence
  int tokens, seqs;
  bool bf16;
  bool wide;              // rows of k and v are 16-byte aligned
  hipStream_t stream;
};
hipError_t launch_kv_append(const KvAppendArgs& a);

}  // namespace mxq
