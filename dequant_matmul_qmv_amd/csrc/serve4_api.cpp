// extern "C" entry points of the operators from the fused projection to attention
// over the 4-bit cache: argument validation before any launch, and dispatch.
#include <hip/hip_runtime.h>

#include <string>

#include "../../include/mxq.h"
#include "serve_checks.h"

using namespace mxq::checks;
using mxq::report;

namespace {

// `rotation` of heads of `dim` values; positions may be null where the call has places
mxq_status check_rotation(const std::string& f, const mxq_rotation* r, int64_t tokens, int dim, mxq_dtype dtype, bool places,
                          mxq::TurnArgs* out) {
  if (!r) return report(MXQ_ERR_INVALID_ARG, f + ": rotation is null");
  if (r->rot < 0) return report(MXQ_ERR_INVALID_ARG, f + ": rot must be >= 0");
  if (r->rot % 2 != 0 || r->rot > dim) return report(MXQ_ERR_UNSUPPORTED, f + ": rot must be even and at most dim");
  if (r->axes < 1 || r->axes > 65536) return report(MXQ_ERR_INVALID_ARG, f + ": axes must be 1 to 2^16");
  if (!(r->eps >= 0.0 && r->eps - r->eps == 0.0)) return report(MXQ_ERR_INVALID_ARG, f + ": eps must be finite and >= 0");
  if ((r->q_weight || r->k_weight) && r->weight_dtype != MXQ_F32 && r->weight_dtype != dtype)
    return report(MXQ_ERR_UNSUPPORTED, f + ": weights must be MXQ_F32 or of the type of q and k");
  if (r->rot > 0 && tokens > 0) {
    if (!r->inv_freq || (!r->positions && !places)) return report(MXQ_ERR_INVALID_ARG, f + ": null inv_freq or positions");
    if (r->positions && r->axes > 1 && r->position_stride < tokens)
      return report(MXQ_ERR_INVALID_ARG, f + ": rows of positions overlap (position_stride < tokens)");
  }
  if (!aligned(r->inv_freq, 4) || !aligned(r->positions, 4) || !aligned(r->axis, 4))
    return report(MXQ_ERR_MISALIGNED, f + ": inv_freq, positions and axis must be 4-byte aligned");
  const uintptr_t w = r->weight_dtype == MXQ_F32 ? 4 : 2;
  if (!aligned(r->q_weight, w) || !aligned(r->k_weight, w))
    return report(MXQ_ERR_MISALIGNED, f + ": weights must be aligned to their elements");
  out->inv_freq = r->inv_freq;
  out->positions = r->positions;
  out->axis_stride = r->axes > 1 ? r->position_stride : 0;
  out->axis = r->axes > 1 ? r->axis : nullptr;
  out->axes = r->axes;
  out->rot = r->rot;
  out->interleaved = r->interleaved != 0;
  out->weight[0] = r->q_weight;
  out->weight[1] = r->k_weight;
  out->weight_f32 = r->weight_dtype == MXQ_F32;
  out->weight_wide = aligned(r->q_weight, 16) && aligned(r->k_weight, 16);
  out->eps = r->eps;
  out->inv_dim = dim > 0 ? 1.0 / dim : 0.0;
  return MXQ_OK;
}

bool rows16(const void* p, int64_t token, int64_t head) { return aligned(p, 16) && ((token | head) & 7) == 0; }

template <typename Args, typename Cache, typename Launch>
mxq_status rope_append(const char* who, const Cache* cache, const void* q, int64_t q_token, int64_t q_head, void* q_out,
                       int64_t q_out_token, int64_t q_out_head, const void* k, int64_t k_token, int64_t k_head, const void* v,
                       int64_t v_token, int64_t v_head, const mxq_rotation* rotation, const int32_t* table,
                       int64_t table_stride, int64_t width, const int32_t* lens, const int32_t* starts, int64_t tokens,
                       int64_t seqs, int heads, mxq_dtype dtype, void* stream, bool plain, Launch launch) {
  const std::string f = who;
  Args a{};
  mxq_status st = check_pool(f, cache, &a.pool);
  if (st != MXQ_OK) return st;
  if (!half_type(dtype)) return report(MXQ_ERR_UNSUPPORTED, f + ": q, k and v must be MXQ_F16 or MXQ_BF16");
  if (heads < 0) return report(MXQ_ERR_INVALID_ARG, f + ": heads must be >= 0");
  if (heads > 65535) return report(MXQ_ERR_UNSUPPORTED, f + ": heads must be below 2^16");
  if (heads > 0 && (a.pool.kv_heads == 0 || heads % a.pool.kv_heads != 0))
    return report(MXQ_ERR_UNSUPPORTED, f + ": heads must be a multiple of the cache's kv_heads");
  st = check_paging(f, a.pool, table, table_stride, width, lens, starts, tokens, seqs);
  if (st != MXQ_OK) return st;
  a.turn.axes = 1;
  if (rotation || !plain) {
    st = check_rotation(f, rotation, tokens, a.pool.dim, dtype, true, &a.turn);
    if (st != MXQ_OK) return st;
  } else if (heads > 0) {
    return report(MXQ_ERR_INVALID_ARG, f + ": rotation is null with query heads to turn");
  }
  // without pages there is still q to turn
  if (tokens == 0 || seqs == 0 || a.pool.kv_heads == 0 || ((width == 0 || a.pool.blocks == 0) && heads == 0)) return MXQ_OK;
  if (!k || !v || (heads > 0 && (!q || !q_out))) return report(MXQ_ERR_INVALID_ARG, f + ": null pointer");
  if (!aligned(q, 2) || !aligned(q_out, 2) || !aligned(k, 2) || !aligned(v, 2))
    return report(MXQ_ERR_MISALIGNED, f + ": q, q_out, k and v must be 2-byte aligned");
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
  a.wide = rows16(k, k_token, k_head) && rows16(v, v_token, v_head);
  a.stream = static_cast<hipStream_t>(stream);
  a.q = mxq::RopeSide{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_token, q_head, q_out_token, q_out_head, heads};
  a.q_wide = rows16(q, q_token, q_head) && rows16(q_out, q_out_token, q_out_head);
  return finish(who, launch(a));
}

}  // namespace

extern "C" {

mxq_status mxq_norm_rope(const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                         int64_t k_head, void* q_out, int64_t q_out_token, int64_t q_out_head, void* k_out,
                         int64_t k_out_token, int64_t k_out_head, const mxq_rotation* rotation, int64_t tokens,
                         int heads, int kv_heads, int dim, mxq_dtype dtype, void* stream) {
  mxq::clear_error();
  if (tokens < 0 || heads < 0 || kv_heads < 0 || dim < 0)
    return report(MXQ_ERR_INVALID_ARG, "mxq_norm_rope: sizes must be >= 0");
  if (!half_type(dtype)) return report(MXQ_ERR_UNSUPPORTED, "mxq_norm_rope: q and k must be MXQ_F16 or MXQ_BF16");
  if (dim > 256) return report(MXQ_ERR_UNSUPPORTED, "mxq_norm_rope: dim must be at most 256");
  if (tokens > INT32_MAX || heads > 65535 || kv_heads > 65535)
    return report(MXQ_ERR_UNSUPPORTED, "mxq_norm_rope: tokens must be below 2^31, heads below 2^16");
  mxq::NormRopeArgs a{};
  const mxq_status st = check_rotation("mxq_norm_rope", rotation, tokens, dim, dtype, false, &a.turn);
  if (st != MXQ_OK) return st;
  if (tokens == 0 || dim == 0 || heads + kv_heads == 0) return MXQ_OK;
  if ((heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)))
    return report(MXQ_ERR_INVALID_ARG, "mxq_norm_rope: null pointer");
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(q_out, 2) || !aligned(k_out, 2))
    return report(MXQ_ERR_MISALIGNED, "mxq_norm_rope: q, k and their outputs must be 2-byte aligned");
  a.side[0] = mxq::RopeSide{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_token, q_head,
                            q_out_token, q_out_head, heads};
  a.side[1] = mxq::RopeSide{static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_token, k_head,
                            k_out_token, k_out_head, kv_heads};
  a.tokens = tokens;
  a.dim = dim;
  a.bf16 = dtype == MXQ_BF16;
  a.stream = static_cast<hipStream_t>(stream);
  return finish("mxq_norm_rope", mxq::launch_norm_rope(a));
}

mxq_status mxq_rope_append(const mxq_kv_cache* cache, const void* q, int64_t q_token, int64_t q_head, void* q_out,
                           int64_t q_out_token, int64_t q_out_head, const void* k, int64_t k_token, int64_t k_head,
                           const void* v, int64_t v_token, int64_t v_head, const mxq_rotation* rotation,
                           const int32_t* table, int64_t table_stride, int64_t width, const int32_t* lens,
                           const int32_t* starts, int64_t tokens, int64_t seqs, int heads, mxq_dtype dtype,
                           void* stream) {
  mxq::clear_error();
  return rope_append<mxq::RopeAppendArgs>("mxq_rope_append", cache, q, q_token, q_head, q_out, q_out_token, q_out_head, k, k_token,
                                          k_head, v, v_token, v_head, rotation, table, table_stride, width, lens, starts, tokens,
                                          seqs, heads, dtype, stream, false, mxq::launch_rope_append);
}

mxq_status mxq_rope_append4(const mxq_kv_cache4* cache, const void* q, int64_t q_token, int64_t q_head, void* q_out,
                            int64_t q_out_token, int64_t q_out_head, const void* k, int64_t k_token, int64_t k_head,
                            const void* v, int64_t v_token, int64_t v_head, const mxq_rotation* rotation,
                            const int32_t* table, int64_t table_stride, int64_t width, const int32_t* lens,
                            const int32_t* starts, int64_t tokens, int64_t seqs, int heads, mxq_dtype dtype,
                            void* stream) {
  mxq::clear_error();
  return rope_append<mxq::RopeAppend4Args>("mxq_rope_append4", cache, q, q_token, q_head, q_out, q_out_token, q_out_head, k, k_token,
                                           k_head, v, v_token, v_head, rotation, table, table_stride, width, lens, starts, tokens,
                                           seqs, heads, dtype, stream, true, mxq::launch_rope_append4);
}

mxq_status mxq_attention4(const void* q, int64_t q_token, int64_t q_head, const mxq_kv_cache4* cache,
                          const int32_t* table, int64_t table_stride, int64_t width, const int32_t* lens,
                          const int32_t* starts, int64_t tokens, int64_t seqs, int heads, int64_t window,
                          float scale, void* out, float* lse, mxq_dtype dtype, void* stream) {
  mxq::clear_error();
  return attention<mxq::Attend4Args>("mxq_attention4", q, q_token, q_head, cache, table, table_stride, width, lens, starts, tokens,
                                     seqs, heads, window, scale, out, lse, dtype, stream, mxq::launch_attend4);
}

}  // extern "C"
