// C ABI of the paged-cache operators (rotary append, decode over an 8-bit
// cache, sliding-window attention): argument checks and launches.  Declared
// in include/seer.h.
#include <cmath>

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

// Pool tensor map of an 8-bit cache: dims (D, head, token, page) or (D, token,
// head, page), whichever lists the smaller stride first; box = one head's 64
// tokens of 128 bytes, 128-byte swizzle.
seer_status make_code_map(const void* base, const seer_dims* d, int token_inner,
                          CUtensorMap* map) {
  auto enc = tensor_map_encoder();
  if (!enc) return SEER_ERR_CUDA;
  const cuuint64_t heads = (cuuint64_t)d->num_kv_heads, tokens = (cuuint64_t)d->block_size;
  const cuuint64_t sh = (cuuint64_t)d->stride_head, st = (cuuint64_t)d->stride_token;
  const cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, token_inner ? tokens : heads,
                              token_inner ? heads : tokens, (cuuint64_t)d->num_pages};
  const cuuint64_t strides[3] = {token_inner ? st : sh, token_inner ? sh : st,
                                 (cuuint64_t)d->stride_page};
  const cuuint32_t box[4] = {(cuuint32_t)kHeadDim, token_inner ? (cuuint32_t)kTileTokens : 1u,
                             token_inner ? 1u : (cuuint32_t)kTileTokens, 1u};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SEER_OK : SEER_ERR_UNSUPPORTED;
}

constexpr int kWPTileRows = 128;  // (token, head) rows of a prefill MMA tile

// Packed query rows [T][Hq][D]: dims (D, head, token); box = 64 dims x the
// group's heads x ntok tokens, 128-byte swizzle.
seer_status make_rows_map(const uint16_t* q, const seer_dims* d, int T, int ntok,
                          CUtensorMap* map) {
  auto enc = tensor_map_encoder();
  if (!enc) return SEER_ERR_CUDA;
  const cuuint64_t row = (cuuint64_t)kHeadDim * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)d->num_q_heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {row, row * d->num_q_heads};
  const cuuint32_t box[3] = {64, (cuuint32_t)(d->num_q_heads / d->num_kv_heads),
                             (cuuint32_t)ntok};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(q), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SEER_OK : SEER_ERR_UNSUPPORTED;
}

constexpr int kClusterMax = 8;  // CTAs that join one row's pieces without a partial

// Pieces per row: the number for which the SMs' resident CTAs are through
// soonest, by waves of CTAs x (a piece's stages + kPieceStart) x (0.6 + 0.4 x the
// share of CTA slots those waves fill), and kCombineStages where partials need
// a combine.  A stage of a lone CTA takes 0.41 us; a piece's start and join
// (launch, three dependent loads, the first copy, the cluster) about 11 of
// them.  Measured, pieces 1 / 2 / 3 / 4 / 8 (us):
//   128 rows of 52 stages, e4m3     30.1 / 28.5 / 28.2 / 37.3 / 40.9   rule: 3
//   256 rows of 58, e4m3            51.3 / 67.9 / 57.1 / 62.0          rule: 1
//   512 rows of 58, e4m3           126.8 / 106.2 / 104.9 / 108.1       rule: 2
//   512 ragged rows to 104, int8   116.5 / 106.6 / 113.8 / 121.6       rule: 2
//   512 ragged rows to 66, bf16      146 / 157 / 160 / 164 / 205       rule: 1
//   1 row of 8, e4m3                 8.5 / 7.1 / 6.7 / 5.8 / 5.1       rule: 8
// (the window's helper does not know the cache type and takes bf16's two CTAs per
// SM, also for 8-bit caches, of which three fit)
constexpr int kPieceStart = 11, kCombineStages = 5;

int ctas_per_sm(const seer_dims* d, int cache) {
  return cache == SEER_CACHE_BF16 || d->num_q_heads / d->num_kv_heads > 8 ? 2 : 3;
}

// Whether the rows go out longest sequence first: where they do not all fit on
// the SMs at once, so that the last to start are short (64 ragged sequences of 4K
// to 32K x 8 heads, int8: 6 us less than the 112 in the order they come).  Ranking costs a
// CTA half a microsecond, which window rows, mostly as long as the window, do
// not get back (147.5 against 146.9).
bool longest_first(const seer_dims* d, int32_t splits, int per_sm) {
  const int64_t ctas = (int64_t)d->batch * d->num_kv_heads * splits;
  return d->batch > 1 && d->batch <= kRankedBatch && ctas > (int64_t)num_sms_current() * per_sm;
}

int32_t pick_splits(const seer_dims* d, int64_t stages, int ctas_per_sm) {
  const int64_t rows = (int64_t)d->batch * d->num_kv_heads;
  const int64_t slots = (int64_t)num_sms_current() * ctas_per_sm;
  int32_t best = 1;
  double least = 1e300;
  for (int32_t s = 1; s <= kMaxSplits; s += s < kClusterMax ? 1 : kClusterMax) {
    const int64_t waves = (rows * s + slots - 1) / slots;
    const double fill = (double)(rows * s) / (double)(waves * slots);
    const double cost = (double)(waves * ((stages + s - 1) / s + kPieceStart)) * (0.6 + 0.4 * fill) +
                        (s > kClusterMax ? kCombineStages : 0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

// Stages of 64 tokens that the longest row of a window with sinks can have.
int64_t window_stages(const seer_dims* d, int32_t window, int32_t sinks) {
  int64_t blocks = ((int64_t)sinks + d->block_size - 1) / d->block_size +
                   ((int64_t)window + d->block_size - 2) / d->block_size + 1;
  if (blocks > d->max_blocks) blocks = d->max_blocks;
  return blocks * (d->block_size / kTileTokens);
}

size_t split_bytes(const seer_dims* d, int32_t splits) {
  if (splits <= kClusterMax) return 0;
  const size_t parts = (size_t)d->batch * d->num_q_heads * (splits / kClusterMax);
  return round256(parts * kHeadDim * sizeof(float)) + round256(parts * sizeof(float));
}

// Checks, tensor maps and parameters of both decode forms, then the launch.
seer_status cache_decode(const seer_dims* d, const seer_cache_attn_args* a, bool window,
                         seer_stream stream) {
  SEER_TRY(check_dims(d));
  if (a == nullptr || !a->q || !a->seqlens || !a->out) return SEER_ERR_INVALID_ARG;
  SEER_TRY(check_cache(d, a->cache_type, a->k_pool, a->v_pool, a->k_scale, a->v_scale));
  if (window) {
    if (a->window < 1 || a->sinks < 0) return SEER_ERR_INVALID_ARG;
  } else {
    if (a->cache_type == SEER_CACHE_BF16) return SEER_ERR_UNSUPPORTED;  // seer_sparse_decode
    if (!a->idx || !a->n_sel || a->k_max < 1 || a->k_max > d->max_blocks)
      return SEER_ERR_INVALID_ARG;
  }
  const int32_t S = a->num_splits;
  if (S < 1 || S > kMaxSplits || (S > kClusterMax && S % kClusterMax)) return SEER_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->out, 2)) return SEER_ERR_UNSUPPORTED;
  if ((int64_t)d->batch * d->num_kv_heads * S > INT_MAX) return SEER_ERR_UNSUPPORTED;
  const size_t need = split_bytes(d, S);
  if (need > 0 && (a->workspace == nullptr || !aligned(a->workspace, 256) ||
                   a->workspace_bytes < need))
    return SEER_ERR_WORKSPACE;
  CacheDecodeParams p = {};
  p.token_inner = d->stride_token < d->stride_head ? 1 : 0;
  CUtensorMap tk, tv;
  if (a->cache_type == SEER_CACHE_BF16) {
    SEER_TRY(make_kv_map(static_cast<const uint16_t*>(a->k_pool), d, p.token_inner, &tk));
    SEER_TRY(make_kv_map(static_cast<const uint16_t*>(a->v_pool), d, p.token_inner, &tv));
  } else {
    SEER_TRY(make_code_map(a->k_pool, d, p.token_inner, &tk));
    SEER_TRY(make_code_map(a->v_pool, d, p.token_inner, &tv));
  }
  p.q = a->q;
  p.page_table = a->page_table;
  p.seqlens = a->seqlens;
  p.idx = a->idx;
  p.n_sel = a->n_sel;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.out = a->out;
  p.lse_out = a->lse_out;
  p.status = a->dev_status;
  p.B = d->batch;
  p.Hq = d->num_q_heads;
  p.Hkv = d->num_kv_heads;
  p.G = d->num_q_heads / d->num_kv_heads;
  p.bs = d->block_size;
  p.max_blocks = d->max_blocks;
  p.k_max = a->k_max;
  // more than a cache can hold sees no more (and keeps positions in 32 bits)
  const int32_t capacity = d->max_blocks * d->block_size;
  p.window = a->window < capacity ? a->window : capacity;
  p.sinks = a->sinks < capacity ? a->sinks : capacity;
  p.S = S;
  p.C = S < kClusterMax ? S : kClusterMax;
  p.num_pages = d->num_pages;
  p.scale_log2 = a->softmax_scale * kLog2e;
  p.by_length = !window && longest_first(d, S, ctas_per_sm(d, a->cache_type));
  if (S > p.C) {
    const size_t parts = (size_t)d->batch * d->num_q_heads * (S / p.C);
    p.o_part = static_cast<float*>(a->workspace);
    p.lse_part = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) +
                                          round256(parts * kHeadDim * sizeof(float)));
  }
  SEER_CUDA(run_cache_decode(tk, tv, p, a->cache_type, window, stream));
  if (S > p.C) {
    CombineParams c = {};
    c.o_part = p.o_part;
    c.lse_part = p.lse_part;
    c.out = a->out;
    c.lse_out = a->lse_out;
    c.S = S / p.C;
    SEER_CUDA(run_combine(c, d->batch, d->num_q_heads, stream, true));
  }
  return SEER_OK;
}

}  // namespace

extern "C" {

int32_t seer_sparse_decode_q8_splits(const seer_dims* d, int32_t k_max) {
  if (check_dims(d) != SEER_OK || k_max < 1) return 1;
  return pick_splits(d, (int64_t)k_max * (d->block_size / kTileTokens),
                     ctas_per_sm(d, SEER_CACHE_E4M3));
}

int32_t seer_window_decode_splits(const seer_dims* d, int32_t window, int32_t sinks) {
  if (check_dims(d) != SEER_OK || window < 1 || sinks < 0) return 1;
  return pick_splits(d, window_stages(d, window, sinks), 2);
}

size_t seer_split_workspace_bytes(const seer_dims* d, int32_t num_splits) {
  if (check_dims(d) != SEER_OK || num_splits < 1 || num_splits > kMaxSplits) return 0;
  return split_bytes(d, num_splits);
}

seer_status seer_sparse_decode_q8(const seer_dims* d, const seer_cache_attn_args* a,
                                  seer_stream stream) {
  NvtxRange range("seer_sparse_decode_q8");
  return cache_decode(d, a, false, stream);
}

seer_status seer_window_decode(const seer_dims* d, const seer_cache_attn_args* a,
                               seer_stream stream) {
  NvtxRange range("seer_window_decode");
  return cache_decode(d, a, true, stream);
}

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
  SEER_CUDA(run_append_rope(p, a->cache_type, num_sms_current(), stream));
  return SEER_OK;
}

seer_status seer_window_prefill(const seer_dims* d, const seer_window_prefill_args* a,
                                seer_stream stream) {
  NvtxRange range("seer_window_prefill");
  SEER_TRY(check_dims(d));
  if (a == nullptr || !a->seqlens) return SEER_ERR_INVALID_ARG;
  if (a->total_tokens < 0 || a->max_new < 1) return SEER_ERR_INVALID_ARG;
  if (a->total_tokens > 0 && (!a->q || !a->out)) return SEER_ERR_INVALID_ARG;
  if (a->cu_tokens == nullptr && (a->total_tokens != d->batch || a->max_new != 1))
    return SEER_ERR_INVALID_ARG;
  if (a->window < 1 || a->sinks < 0) return SEER_ERR_INVALID_ARG;
  if (!(a->softmax_scale > 0.f) || !(a->softmax_scale < INFINITY)) return SEER_ERR_INVALID_ARG;
  SEER_TRY(check_cache(d, SEER_CACHE_BF16, a->k_pool, a->v_pool, nullptr, nullptr));
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return SEER_ERR_UNSUPPORTED;
  if (a->total_tokens == 0) return SEER_OK;
  WindowPrefillParams p = {};
  p.cu = a->cu_tokens;
  p.seqlens = a->seqlens;
  p.page_table = a->page_table;
  p.out = a->out;
  p.lse = a->lse_out;
  p.status = a->dev_status;
  p.B = d->batch;
  p.Hq = d->num_q_heads;
  p.Hkv = d->num_kv_heads;
  p.G = d->num_q_heads / d->num_kv_heads;
  p.bs = d->block_size;
  p.max_blocks = d->max_blocks;
  p.T = a->total_tokens;
  p.max_new = a->max_new;
  // more than a cache can hold sees no more (and keeps positions in 32 bits)
  const int32_t capacity = d->max_blocks * d->block_size;
  p.window = a->window < capacity ? a->window : capacity;
  p.sinks = a->sinks < capacity ? a->sinks : capacity;
  p.ntok = kWPTileRows / p.G;
  p.v_pool = a->v_pool;
  p.stride_page = d->stride_page;
  p.stride_token = d->stride_token;
  p.stride_head = d->stride_head;
  p.token_inner = d->stride_token < d->stride_head ? 1 : 0;
  p.num_pages = d->num_pages;
  p.scale_log2 = a->softmax_scale * kLog2e;
  CUtensorMap tq, tk, tv;
  SEER_TRY(make_rows_map(a->q, d, p.T, p.ntok, &tq));
  SEER_TRY(make_kv_map(a->k_pool, d, p.token_inner, &tk));
  SEER_TRY(make_kv_map(a->v_pool, d, p.token_inner, &tv));
  SEER_CUDA(run_window_prefill(tq, tk, tv, p, num_sms_current(), stream));
  return SEER_OK;
}

}  // extern "C"
