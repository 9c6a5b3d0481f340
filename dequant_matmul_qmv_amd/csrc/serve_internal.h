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

// A launch holds less than 2^32 threads in its grid's first dimension.  Calls
// that need more give kTooLarge, with nothing enqueued.
constexpr hipError_t kTooLarge = hipErrorInvalidConfiguration;
inline bool grid_fits(int64_t workgroups, int threads) { return workgroups < (int64_t{1} << 32) / threads; }

// Runs `enqueue(workspace)` with `bytes` of device memory that stay the
// stream's own until what it enqueues is done: the split workspace cache
// (workspace.cpp), or, on a stream being captured, memory of the graph.
// hipErrorOutOfMemory, with nothing enqueued, where none can be had.
template <typename F>
hipError_t with_split_workspace(const DeviceInfo& dev, hipStream_t stream, size_t bytes, F enqueue) {
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(stream, &cap) != hipSuccess) {
    (void)hipGetLastError();
    cap = hipStreamCaptureStatusNone;
  }
  if (cap == hipStreamCaptureStatusNone) {
    std::lock_guard<std::mutex> lk(split_workspace_mutex());
    float* ws = split_workspace_locked(dev.device, stream, bytes);
    return ws == nullptr ? hipErrorOutOfMemory : enqueue(ws);
  }
  void* ws = nullptr;
  if (hipMallocAsync(&ws, bytes, stream) != hipSuccess) {
    (void)hipGetLastError();
    return hipErrorOutOfMemory;
  }
  const hipError_t e = enqueue(static_cast<float*>(ws)), f = hipFreeAsync(ws, stream);
  return e != hipSuccess ? e : f;
}

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

// Attention of new tokens over the cache.  Partial results of a key range, one
// slot a workgroup: rows of dim f32 means, then their maxima and weights.
struct AttendArgs {
  KvPool pool;
  const uint16_t* q;
  int64_t q_token, q_head;
  uint16_t* out;          // [tokens, heads, dim]
  float* lse;             // [tokens, heads] or null
  const int32_t* table;
  int64_t table_stride;
  int width;
  const int32_t* lens;
  const int32_t* starts;  // null: one token for each sequence
  int tokens, seqs, heads, group;  // group: query heads of one kv head
  int window;             // 0: none
  float scale2;           // softmax scale times log2(e)
  bool bf16;
  hipStream_t stream;
  // set by the launcher
  float* part;            // means [slots, rows, dim]
  float* part_ml;         // (maximum, weight) [slots, rows, 2]
  int slots;              // of them
  int target;             // workgroups the few-row work is split for
  int min_chunks;         // least 64-key chunks of a part
  int few_rows;           // most rows (new tokens times group) of a sequence that the few-row kernel takes
  int join_new;           // most new tokens of such a sequence
  float* many_part;       // the same of the many-row kernel
  float* many_ml;
  int many_splits;        // parts of its key axis
  int many_units;         // workgroups
};
// The many-row kernel (attend_many.hip): its tiles at most, the bytes of its
// partial results, its launch (with the second one that joins them).
int64_t many_tiles(const AttendArgs& a);
size_t many_part_bytes(const AttendArgs& a);
hipError_t launch_many(const AttendArgs& a, float* ws);
hipError_t launch_attend(const AttendArgs& a, const DeviceInfo& dev);

// What sampling's kernels leave of a row for the later ones.
struct SamplePlan {
  int state;
  uint32_t top;
  uint32_t low;  // no kept token's key is below
  float scale;   // bins a unit of logit
  uint32_t listed, arrived;
  double total;  // the row's weight, in the integers' unit; without top_k
};

// One draw for each row of logits.  Settings: arrays of a value for each row,
// or (null) one value for all.
struct SampleArgs {
  const void* logits;
  int64_t row_stride;  // elements
  int rows, vocab;
  int type;            // mxq_dtype value
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all;
  int top_k_all;
  float top_p_all, min_p_all;
  int32_t* tokens;
  float* probs;
  hipStream_t stream;
  // set by the launcher
  uint32_t* cells;     // largest key of each 64 tokens [rows, cell_count]
  double* pieces;      // weight of each 512 tokens [rows, piece_count]
  int cell_count, piece_count;
  // of rows whose kept tokens are more than a list (null where none can be)
  SamplePlan* plans;
  unsigned long long* bin_mass;  // weight of each bin by value [rows, 2048]
  uint32_t* bin_count;
  unsigned long long* list;      // tokens of the bins in which the prefix ends [rows, 2048]
  unsigned long long* kept;      // kept weight of each piece but for the list's [rows, piece_count]
  int span;            // tokens of a workgroup, a multiple of 8192
  bool ahead;          // bins are filled beside the draw
};
hipError_t launch_sample(const SampleArgs& a, const DeviceInfo& dev);

}  // namespace mxq
