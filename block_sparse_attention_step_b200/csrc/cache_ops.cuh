// Parameter blocks and launchers of the paged-cache operators: rotary append,
// decode over an 8-bit cache, sliding-window attention (internal).
#pragma once

#include "seer_kernels.cuh"

namespace seer {

// Rotary append of a ragged batch's new tokens to the paged cache.
struct AppendParams {
  const uint16_t* q;  // optional
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  const int32_t* cu;         // [B + 1], or nullptr: one token per sequence
  const int32_t* positions;  // optional [T]
  const int32_t* seqlens;
  const int32_t* page_table;
  const float* rope;  // [max_position][rot], nullptr when rot == 0
  uint16_t* q_out;
  void* k_pool;
  void* v_pool;
  float* k_scale;  // [num_pages][Hkv], 8-bit cache
  float* v_scale;
  float* kbar;  // optional
  int32_t* status;
  int B, Hq, Hkv, bs, max_blocks, T, max_new, max_position, rot, interleaved;
  int64_t num_pages, stride_page, stride_token, stride_head;
  // set by the launcher
  int rows_kv;      // the row role writes k and v too (bf16, no pooled keys)
  int tile_tokens;  // tokens of a row-role tile
  int segments, segment_rows;  // parts a token's rows are cut into, one warp each
  int heads;        // KV heads of a block per CTA (divides Hkv)
  uint64_t block_share;  // 2^32 x block CTAs / all CTAs, rounded up
};

cudaError_t run_append_rope(AppendParams p, int cache, int num_sms, cudaStream_t stream);
cudaError_t run_rope_table(float* table, int max_position, int rot, double base,
                           cudaStream_t stream);

constexpr int kRankedBatch = 256;

// Decode attention over a block list or a window with sinks.
struct CacheDecodeParams {
  const uint16_t* q;  // [B][Hq][D]
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* idx;    // [B][Hkv][k_max], list form
  const int32_t* n_sel;  // [B][Hkv]
  const float* k_scale;  // [num_pages][Hkv], 8-bit cache
  const float* v_scale;
  float* o_part;  // [B][Hq][S / C][D] when S > C, else nullptr
  float* lse_part;
  uint16_t* out;
  float* lse_out;  // optional
  int32_t* status;
  int B, Hq, Hkv, G, bs, max_blocks, k_max, window, sinks;
  int S, C;         // pieces per row, CTAs per cluster (C = min(S, 8), divides S)
  int token_inner;  // tensor map dims are (D, token, head, page), not (D, head, token, page)
  int by_length;    // longest sequences first (B <= kRankedBatch)
  int64_t num_pages;
  float scale_log2;
};

// Sliding-window attention of a ragged chunk of query tokens.
struct WindowPrefillParams {
  const int32_t* cu;  // [B + 1], or nullptr: one token per sequence
  const int32_t* seqlens;
  const int32_t* page_table;
  const uint16_t* v_pool;
  uint16_t* out;  // [T][Hq][D]
  float* lse;     // optional [Hq][T]
  int32_t* status;
  int B, Hq, Hkv, G, bs, max_blocks, T, max_new, window, sinks;
  int ntok;  // query tokens of a 128-row tile, floor(128 / G)
  int token_inner;
  int64_t num_pages, stride_page, stride_token, stride_head;
  float scale_log2;
};

cudaError_t run_window_prefill(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const WindowPrefillParams& p, int num_sms, cudaStream_t stream);

cudaError_t run_cache_decode(const CUtensorMap& tk, const CUtensorMap& tv,
                             const CacheDecodeParams& p, int cache, bool window,
                             cudaStream_t stream);

}  // namespace seer
