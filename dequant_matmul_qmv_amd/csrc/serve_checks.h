// Argument checks shared by the serving operators' entry points, and attention's call
// over either form of the cache.
#pragma once

#include <string>

#include "serve_internal.h"

namespace mxq {
namespace checks {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline mxq_status finish(const char* who, hipError_t e) {
  if (e == kTooLarge)
    return report(MXQ_ERR_UNSUPPORTED, std::string(who) + ": more sequences, tokens and heads than one launch holds (split the call)");
  return e == hipSuccess ? MXQ_OK : report_hip(who, e);
}

inline bool half_type(mxq_dtype t) { return t == MXQ_F16 || t == MXQ_BF16; }

// Sizes and pointers of a cache of either form; the scales' alignment in bytes.
template <typename Cache>
mxq_status check_cache(const std::string& f, const Cache* c, uintptr_t scales, const char* rule) {
  if (!c) return report(MXQ_ERR_INVALID_ARG, f + ": cache is null");
  if (c->blocks < 0 || c->kv_heads < 0) return report(MXQ_ERR_INVALID_ARG, f + ": blocks and kv_heads must be >= 0");
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return report(MXQ_ERR_UNSUPPORTED, f + ": block must be 16, 32, 64 or 128");
  if (c->dim != 64 && c->dim != 128) return report(MXQ_ERR_UNSUPPORTED, f + ": dim must be 64 or 128");
  if (c->blocks > INT32_MAX || c->kv_heads > 65535)
    return report(MXQ_ERR_UNSUPPORTED, f + ": blocks must be below 2^31, kv_heads below 2^16");
  if (c->blocks > 0 && c->kv_heads > 0) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return report(MXQ_ERR_INVALID_ARG, f + ": null cache pointer");
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, scales) || !aligned(c->v_scale, scales))
      return report(MXQ_ERR_MISALIGNED, f + rule);
  }
  return MXQ_OK;
}

inline mxq_status check_pool(const std::string& f, const mxq_kv_cache* c, KvPool* out) {
  const mxq_status st = check_cache(f, c, 4, ": cache codes must be 16-byte, scales 4-byte aligned");
  if (st != MXQ_OK) return st;
  *out = KvPool{c->k, c->v, c->k_scale, c->v_scale, c->blocks, c->kv_heads, c->block, c->dim};
  return MXQ_OK;
}

inline mxq_status check_pool(const std::string& f, const mxq_kv_cache4* c, KvPool4* out) {
  const mxq_status st = check_cache(f, c, 16, ": cache words and scales must be 16-byte aligned");
  if (st != MXQ_OK) return st;
  *out = KvPool4{c->k, c->v, c->k_scale, c->v_scale, c->blocks, c->kv_heads, c->block, c->dim};
  return MXQ_OK;
}

// table, lens and starts of the calls on a paged cache
template <typename Pool>
mxq_status check_paging(const std::string& f, const Pool& pool, const int32_t* table, int64_t table_stride,
                        int64_t width, const int32_t* lens, const int32_t* starts, int64_t tokens, int64_t seqs) {
  if (tokens < 0 || seqs < 0 || width < 0) return report(MXQ_ERR_INVALID_ARG, f + ": tokens, seqs and width must be >= 0");
  if (!starts && tokens != seqs)
    return report(MXQ_ERR_INVALID_ARG, f + ": without starts every sequence has one token (tokens == seqs)");
  if (tokens > (int64_t{1} << 24) || seqs > (int64_t{1} << 24))
    return report(MXQ_ERR_UNSUPPORTED, f + ": tokens and seqs must be at most 2^24");
  if (width > INT32_MAX / pool.block) return report(MXQ_ERR_UNSUPPORTED, f + ": width * block must be below 2^31");
  if (tokens == 0 || seqs == 0) return MXQ_OK;
  if (!lens || (width > 0 && !table)) return report(MXQ_ERR_INVALID_ARG, f + ": null table or lens");
  if (seqs > 1 && table_stride < width) return report(MXQ_ERR_INVALID_ARG, f + ": table rows overlap (table_stride < width)");
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4))
    return report(MXQ_ERR_MISALIGNED, f + ": table, lens and starts must be 4-byte aligned");
  return MXQ_OK;
}

// Checks an attention call and launches it.
template <typename Args, typename Cache, typename Launch>
mxq_status attention(const char* who, const void* q, int64_t q_token, int64_t q_head, const Cache* cache, const int32_t* table,
                     int64_t table_stride, int64_t width, const int32_t* lens, const int32_t* starts, int64_t tokens,
                     int64_t seqs, int heads, int64_t window, float scale, void* out, float* lse, mxq_dtype dtype, void* stream,
                     Launch launch) {
  const std::string f = who;
  Args a{};
  mxq_status st = check_pool(f, cache, &a.pool);
  if (st != MXQ_OK) return st;
  if (!half_type(dtype)) return report(MXQ_ERR_UNSUPPORTED, f + ": q must be MXQ_F16 or MXQ_BF16");
  if (heads < 0 || window < 0) return report(MXQ_ERR_INVALID_ARG, f + ": heads and window must be >= 0");
  if (heads > 65535) return report(MXQ_ERR_UNSUPPORTED, f + ": heads must be below 2^16");
  if (heads > 0 && (a.pool.kv_heads == 0 || heads % a.pool.kv_heads != 0))
    return report(MXQ_ERR_UNSUPPORTED, f + ": heads must be a multiple of the cache's kv_heads");
  if (heads == 0) return MXQ_OK;
  // the kernels take it times log2(e)
  const float scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  if (!(scale2 - scale2 == 0.0f)) return report(MXQ_ERR_INVALID_ARG, f + ": scale must be finite, also times log2(e)");
  st = check_paging(f, a.pool, table, table_stride, width, lens, starts, tokens, seqs);
  if (st != MXQ_OK) return st;
  if (tokens == 0 || seqs == 0) return MXQ_OK;
  if (tokens * heads > INT32_MAX) return report(MXQ_ERR_UNSUPPORTED, f + ": tokens * heads must be below 2^31");
  if (!q || !out) return report(MXQ_ERR_INVALID_ARG, f + ": null pointer");
  if (!aligned(q, 16) || ((q_token | q_head) & 7) != 0 || !aligned(out, 8) || !aligned(lse, 4))
    return report(MXQ_ERR_MISALIGNED,
                  f + ": rows of q must be 16-byte, out 8-byte and lse 4-byte aligned");
  a.q = static_cast<const uint16_t*>(q);
  a.q_token = q_token;
  a.q_head = q_head;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.table = table;
  a.table_stride = table_stride;
  a.width = static_cast<int>(width);
  a.lens = lens;
  a.starts = starts;
  a.tokens = static_cast<int>(tokens);
  a.seqs = static_cast<int>(seqs);
  a.heads = heads;
  a.group = heads / a.pool.kv_heads;
  a.window = static_cast<int>(window > INT32_MAX ? 0 : window);
  a.scale2 = scale2;
  a.bf16 = dtype == MXQ_BF16;
  a.stream = static_cast<hipStream_t>(stream);
  DeviceInfo dev;
  const hipError_t e = device_info(&dev);
  return finish(who, e != hipSuccess ? e : launch(a, dev));
}

}  // namespace checks
}  // namespace mxq
