// C ABI of the paged-cache operators (rotary append, decode over an 8-bit
// cache, sliding-window attention): argument checks and launches.  Declared
// in include/seer.h.
#include "api_util.cuh"
#include "cache_ops.cuh"

using namespace seer;

namespace {

// Pools of any cache type; scales present exactly for the 8-bit types.
seer_status check_cache(const seer_dims* d, int cache, const void* k_pool, const void* v_pool,
                        const float* k_scale, const float* v_scale) {
  if (cache != SEER_CACHE_BF16 && cache != SEER_CACHE_E4M3 && cache != SEER_CACHE_INT8)
    return SEER_ERR_INVALID_ARG;
  SEER_TRY(check_pool(d, static_cast<const uint16_t*>(k_pool)));
  SEER_TRY(check_pool(d, static_cast<const uint16_t*>(v_pool)));
  if (cache == SEER_CACHE_BF16) {
    if (k_scale || v_scale) return SEER_ERR_INVALID_ARG;
    return SEER_OK;
  }
  if (!k_scale || !v_scale) return SEER_ERR_INVALID_ARG;
  if (d->stride_page % 16 || d->stride_token % 16 || d->stride_head % 16)
    return SEER_ERR_UNSUPPORTED;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return SEER_ERR_UNSUPPORTED;
  return SEER_OK;
}

}  // namespace

extern "C" {

seer_status seer_rope_table(int32_t max_position, int32_t rotary_dim, double base, float* table,
                            seer_stream stream) {
  if (!table || max_position < 1 || rotary_dim < 2 || rotary_dim % 2 || !(base > 0.0))
    return SEER_ERR_INVALID_ARG;
  if (rotary_dim > kHeadDim || !aligned(table, 4)) return SEER_ERR_UNSUPPORTED;
  SEER_CUDA(run_rope_table(table, max_position, rotary_dim, base, stream));
  return SEER_OK;
}

seer_status seer_append_rope(const seer_dims* d, const seer_append_args* a, seer_stream stream) {
  NvtxRange range("seer_append_rope");
  SEER_TRY(check_dims(d));
  if (a == nullptr || !a->seqlens) return SEER_ERR_INVALID_ARG;
  if (a->total_tokens < 0 || a->max_new < 1) return SEER_ERR_INVALID_ARG;
  // no rows: their pointers may be NULL, as an empty tensor's is
  if (a->total_tokens > 0 && (!a->k_new || !a->v_new)) return SEER_ERR_INVALID_ARG;
  if (a->total_tokens > 0 && (a->q == nullptr) != (a->q_out == nullptr))
    return SEER_ERR_INVALID_ARG;
  if (a->cu_tokens == nullptr && (a->total_tokens != d->batch || a->max_new != 1))
    return SEER_ERR_INVALID_ARG;
  if (a->rotary_dim < 0 || (a->interleaved != 0 && a->interleaved != 1))
    return SEER_ERR_INVALID_ARG;
  if ((a->rope == nullptr) != (a->rotary_dim == 0)) return SEER_ERR_INVALID_ARG;
  if (a->rotary_dim > 0 && a->max_position < 1) return SEER_ERR_INVALID_ARG;
  if (a->rotary_dim % 16 || a->rotary_dim > kHeadDim) return SEER_ERR_UNSUPPORTED;
  SEER_TRY(check_cache(d, a->cache_type, a->k_pool, a->v_pool, a->k_scale, a->v_scale));
  AppendParams p = {};
  p.q_stride = a->q_stride ? a->q_stride : (int64_t)d->num_q_heads * kHeadDim;
  p.k_stride = a->k_stride ? a->k_stride : (int64_t)d->num_kv_heads * kHeadDim;
  p.v_stride = a->v_stride ? a->v_stride : (int64_t)d->num_kv_heads * kHeadDim;
  if (p.q_stride < (int64_t)d->num_q_heads * kHeadDim ||
      p.k_stride < (int64_t)d->num_kv_heads * kHeadDim ||
      p.v_stride < (int64_t)d->num_kv_heads * kHeadDim)
    return SEER_ERR_INVALID_ARG;
  // turned in place, a row stays where it is: q_out then has q's stride
  p.q_out_stride = a->q_out == a->q ? p.q_stride : (int64_t)d->num_q_heads * kHeadDim;
  if (p.q_stride % 8 || p.k_stride % 8 || p.v_stride % 8) return SEER_ERR_UNSUPPORTED;
  if (!aligned(a->q, 16) || !aligned(a->k_new, 16) || !aligned(a->v_new, 16) ||
      !aligned(a->q_out, 16) || !aligned(a->rope, 16) || !aligned(a->kbar, 16))
    return SEER_ERR_UNSUPPORTED;
  p.q = a->q;
  p.k = a->k_new;
  p.v = a->v_new;
  p.cu = a->cu_tokens;
  p.positions = a->positions;
  p.seqlens = a->seqlens;
  p.page_table = a->page_table;
  p.rope = a->rope;
  p.q_out = a->q_out;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.kbar = a->kbar;
  p.status = a->dev_status;
  p.B = d->batch;
  p.Hq = d->num_q_heads;
  p.Hkv = d->num_kv_heads;
  p.bs = d->block_size;
  p.max_blocks = d->max_blocks;
  p.T = a->total_tokens;
  p.max_new = a->max_new;
  p.max_position = a->max_position;
  p.rot = a->rotary_dim;
  p.interleaved = a->interleaved;
  p.num_pages = d->num_pages;
  p.stride_page = d->stride_page;
  p.stride_token = d->stride_token;
  p.stride_head = d->stride_head;
  SEER_CUDA(run_append_rope(p, a->cache_type, stream));
  return SEER_OK;
}

}  // extern "C"
