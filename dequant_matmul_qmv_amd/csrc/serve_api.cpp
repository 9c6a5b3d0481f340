// extern "C" entry points of the serving operators: argument validation
// before any launch, as in api.cpp, and dispatch.
#include <hip/hip_runtime.h>

#include <string>

#include "../../include/mxq.h"
#include "serve_internal.h"

namespace {

using mxq::report;
using mxq::report_hip;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mxq_status finish(const char* who, hipError_t e) {
  if (e == mxq::kTooLarge)
    return report(MXQ_ERR_UNSUPPORTED, std::string(who) + ": more sequences, tokens and heads than one launch holds (split the call)");
  return e == hipSuccess ? MXQ_OK : report_hip(who, e);
}

bool half_type(mxq_dtype t) { return t == MXQ_F16 || t == MXQ_BF16; }

mxq_status check_pool(const std::string& f, const mxq_kv_cache* c, mxq::KvPool* out) {
  if (!c) return report(MXQ_ERR_INVALID_ARG, f + ": cache is null");
  if (c->blocks < 0 || c->kv_heads < 0) return report(MXQ_ERR_INVALID_ARG, f + ": blocks and kv_heads must be >= 0");
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return report(MXQ_ERR_UNSUPPORTED, f + ": block must be 16, 32, 64 or 128");
  if (c->dim != 64 && c->dim != 128) return report(MXQ_ERR_UNSUPPORTED, f + ": dim must be 64 or 128");
  if (c->blocks > INT32_MAX || c->kv_heads > 65535)
    return report(MXQ_ERR_UNSUPPORTED, f + ": blocks must be below 2^31, kv_heads below 2^16");
  if (c->blocks > 0 && c->kv_heads > 0) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return report(MXQ_ERR_INVALID_ARG, f + ": null cache pointer");
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
      return report(MXQ_ERR_MISALIGNED, f + ": cache codes must be 16-byte, scales 4-byte aligned");
  }
  *out = mxq::KvPool{c->k, c->v, c->k_scale, c->v_scale, c->blocks, c->kv_heads, c->block, c->dim};
  return MXQ_OK;
}

// table, lens and starts of the calls on a paged cache
mxq_status check_paging(const std::string& f, const mxq::KvPool& pool, const int32_t* table, int64_t table_stride,
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

}  // namespace

extern "C" {

mxq_status mxq_rope(const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                    int64_t k_head, void* q_out, int64_t q_out_token, int64_t q_out_head, void* k_out,
                    int64_t k_out_token, int64_t k_out_head, const float* inv_freq,
                    const int32_t* positions, int64_t tokens, int heads, int kv_heads, int dim, int rot,
                    int interleaved, mxq_dtype dtype, void* stream) {
  mxq::clear_error();
  if (tokens < 0 || heads < 0 || kv_heads < 0 || dim < 0 || rot < 0)
    return report(MXQ_ERR_INVALID_ARG, "mxq_rope: sizes must be >= 0");
  if (!half_type(dtype)) return report(MXQ_ERR_UNSUPPORTED, "mxq_rope: q and k must be MXQ_F16 or MXQ_BF16");
  if (dim > 256) return report(MXQ_ERR_UNSUPPORTED, "mxq_rope: dim must be at most 256");
  if (rot % 2 != 0 || rot > dim) return report(MXQ_ERR_UNSUPPORTED, "mxq_rope: rot must be even and at most dim");
  if (tokens > INT32_MAX || heads > 65535 || kv_heads > 65535)
    return report(MXQ_ERR_UNSUPPORTED, "mxq_rope: tokens must be below 2^31, heads below 2^16");
  if (tokens == 0 || dim == 0 || heads + kv_heads == 0) return MXQ_OK;
  if ((heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)) || !positions || (rot > 0 && !inv_freq))
    return report(MXQ_ERR_INVALID_ARG, "mxq_rope: null pointer");
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(q_out, 2) || !aligned(k_out, 2) || !aligned(inv_freq, 4) ||
      !aligned(positions, 4))
    return report(MXQ_ERR_MISALIGNED, "mxq_rope: q, k and their outputs must be 2-byte, inv_freq and positions 4-byte aligned");
  mxq::RopeArgs a{};
  a.side[0] = mxq::RopeSide{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_token, q_head,
                            q_out_token, q_out_head, heads};
  a.side[1] = mxq::RopeSide{static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_token, k_head,
                            k_out_token, k_out_head, kv_heads};
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.tokens = tokens;
  a.dim = dim;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.bf16 = dtype == MXQ_BF16;
  a.stream = static_cast<hipStream_t>(stream);
  return finish("mxq_rope", mxq::launch_rope(a));
}

mxq_status mxq_kv_append(const mxq_kv_cache* cache, const void* k, int64_t k_token, int64_t k_head,
                         const void* v, int64_t v_token, int64_t v_head, const int32_t* table,
                         int64_t table_stride, int64_t width, const int32_t* lens, const int32_t* starts,
                         int64_t tokens, int64_t seqs, mxq_dtype dtype, void* stream) {
  mxq::clear_error();
  mxq::KvAppendArgs a{};
  mxq_status st = check_pool("mxq_kv_append", cache, &a.pool);
  if (st != MXQ_OK) return st;
  if (!half_type(dtype)) return report(MXQ_ERR_UNSUPPORTED, "mxq_kv_append: k and v must be MXQ_F16 or MXQ_BF16");
  st = check_paging("mxq_kv_append", a.pool, table, table_stride, width, lens, starts, tokens, seqs);
  if (st != MXQ_OK) return st;
  if (tokens == 0 || seqs == 0 || width == 0 || a.pool.blocks == 0 || a.pool.kv_heads == 0) return MXQ_OK;
  if (!k || !v) return report(MXQ_ERR_INVALID_ARG, "mxq_kv_append: null pointer");
  if (!aligned(k, 2) || !aligned(v, 2)) return report(MXQ_ERR_MISALIGNED, "mxq_kv_append: k and v must be 2-byte aligned");
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.table = table;
  a.table_stride = table_stride;
  a.width = static_cast<int>(width);
  a.lens = lens;
  a.starts = starts;
  a.tokens = static_cast<int>(tokens);
  a.seqs = static_cast<int>(seqs);
  a.bf16 = dtype == MXQ_BF16;
  a.wide = aligned(k, 16) && aligned(v, 16) && ((k_token | k_head | v_token | v_head) & 7) == 0;
  a.stream = static_cast<hipStream_t>(stream);
  return finish("mxq_kv_append", mxq::launch_kv_append(a));
}

mxq_status mxq_attention(const void* q, int64_t q_token, int64_t q_head, const mxq_kv_cache* cache,
                         const int32_t* table, int64_t table_stride, int64_t width, const int32_t* lens,
                         const int32_t* starts, int64_t tokens, int64_t seqs, int heads, int64_t window,
                         float scale, void* out, float* lse, mxq_dtype dtype, void* stream) {
  mxq::clear_error();
  mxq::AttendArgs a{};
  mxq_status st = check_pool("mxq_attention", cache, &a.pool);
  if (st != MXQ_OK) return st;
  if (!half_type(dtype)) return report(MXQ_ERR_UNSUPPORTED, "mxq_attention: q must be MXQ_F16 or MXQ_BF16");
  if (heads < 0 || window < 0) return report(MXQ_ERR_INVALID_ARG, "mxq_attention: heads and window must be >= 0");
  if (heads > 65535) return report(MXQ_ERR_UNSUPPORTED, "mxq_attention: heads must be below 2^16");
  if (heads > 0 && (a.pool.kv_heads == 0 || heads % a.pool.kv_heads != 0))
    return report(MXQ_ERR_UNSUPPORTED, "mxq_attention: heads must be a multiple of the cache's kv_heads");
  if (heads == 0) return MXQ_OK;
  // the kernels take it times log2(e)
  const float scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  if (!(scale2 - scale2 == 0.0f)) return report(MXQ_ERR_INVALID_ARG, "mxq_attention: scale must be finite, also times log2(e)");
  st = check_paging("mxq_attention", a.pool, table, table_stride, width, lens, starts, tokens, seqs);
  if (st != MXQ_OK) return st;
  if (tokens == 0 || seqs == 0) return MXQ_OK;
  if (tokens * heads > INT32_MAX) return report(MXQ_ERR_UNSUPPORTED, "mxq_attention: tokens * heads must be below 2^31");
  if (!q || !out) return report(MXQ_ERR_INVALID_ARG, "mxq_attention: null pointer");
  if (!aligned(q, 16) || ((q_token | q_head) & 7) != 0 || !aligned(out, 8) || !aligned(lse, 4))
    return report(MXQ_ERR_MISALIGNED,
                  "mxq_attention: rows of q must be 16-byte, out 8-byte and lse 4-byte aligned");
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
  mxq::DeviceInfo dev;
  const hipError_t e = mxq::device_info(&dev);
  return finish("mxq_attention", e != hipSuccess ? e : mxq::launch_attend(a, dev));
}

mxq_status mxq_sample(const void* logits, int64_t row_stride, int64_t rows, int64_t vocab, mxq_dtype dtype,
                      const float* u, const mxq_sampling* settings, int32_t* tokens, float* probs, void* stream) {
  mxq::clear_error();
  if (rows < 0 || vocab < 0) return report(MXQ_ERR_INVALID_ARG, "mxq_sample: rows and vocab must be >= 0");
  if (dtype != MXQ_F16 && dtype != MXQ_BF16 && dtype != MXQ_F32)
    return report(MXQ_ERR_UNSUPPORTED, "mxq_sample: logits must be MXQ_F16, MXQ_BF16 or MXQ_F32");
  if (vocab > (1 << 20)) return report(MXQ_ERR_UNSUPPORTED, "mxq_sample: vocab must be at most 2^20");
  if (rows > (1 << 24)) return report(MXQ_ERR_UNSUPPORTED, "mxq_sample: rows must be at most 2^24");
  if (rows == 0) return MXQ_OK;
  if (vocab == 0) return report(MXQ_ERR_INVALID_ARG, "mxq_sample: nothing to draw from (vocab is 0)");
  if (!logits || !u || !settings || !tokens || !probs) return report(MXQ_ERR_INVALID_ARG, "mxq_sample: null pointer");
  if (rows > 1 && row_stride < vocab)
    return report(MXQ_ERR_INVALID_ARG, "mxq_sample: rows overlap (row_stride < vocab)");
  if (!aligned(logits, dtype == MXQ_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(tokens, 4) || !aligned(probs, 4) ||
      !aligned(settings->temperature, 4) || !aligned(settings->top_k, 4) || !aligned(settings->top_p, 4) ||
      !aligned(settings->min_p, 4))
    return report(MXQ_ERR_MISALIGNED, "mxq_sample: a pointer is not aligned to its elements");
  mxq::SampleArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.rows = static_cast<int>(rows);
  a.vocab = static_cast<int>(vocab);
  a.type = static_cast<int>(dtype);
  a.u = u;
  a.temperature = settings->temperature;
  a.top_k = settings->top_k;
  a.top_p = settings->top_p;
  a.min_p = settings->min_p;
  a.temperature_all = settings->temperature_all;
  a.top_k_all = settings->top_k_all;
  a.top_p_all = settings->top_p_all;
  a.min_p_all = settings->min_p_all;
  a.tokens = tokens;
  a.probs = probs;
  a.stream = static_cast<hipStream_t>(stream);
  mxq::DeviceInfo dev;
  const hipError_t e = mxq::device_info(&dev);
  return finish("mxq_sample", e != hipSuccess ? e : mxq::launch_sample(a, dev));
}

}  // extern "C"
