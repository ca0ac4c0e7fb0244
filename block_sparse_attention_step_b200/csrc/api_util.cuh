// Host-side helpers of the C ABI's entry points: argument checks, tensor maps,
// NVTX ranges and error reporting.
#pragma once

#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <climits>
#include <cstdlib>
#include <mutex>

#include "seer_kernels.cuh"

namespace seer {

constexpr int kMaxDevices = 64;

// NVTX ranges around each step and each stage it enqueues, for profilers
// (ncu --nvtx-include, nsys): compiled in, off unless the environment has
// SEER_NVTX=1 when the library first checks (a host-side push/pop only).
inline bool nvtx_on() {
  static const bool on = [] {
    const char* v = std::getenv("SEER_NVTX");
    return v != nullptr && v[0] == '1';
  }();
  return on;
}

struct NvtxRange {
  const bool on;
  explicit NvtxRange(const char* name) : on(nvtx_on()) {
    if (on) nvtxRangePushA(name);
  }
  ~NvtxRange() {
    if (on) nvtxRangePop();
  }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

inline int num_sms_current() {
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < kMaxDevices) {
    const int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 148;
  if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Pool tensor map: dims (D, head, token, page) or (D, token, head, page),
// whichever lists the smaller stride first; box = 64 dims x 64 tokens,
// 128-byte swizzle (conflict-free ldmatrix rows).
inline seer_status make_kv_map(const uint16_t* base, const seer_dims* d, int token_inner, CUtensorMap* map) {
  auto enc = tensor_map_encoder();
  if (!enc) return SEER_ERR_CUDA;
  cuuint64_t dims[4];
  cuuint64_t strides[3];
  cuuint32_t box[4];
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  dims[0] = (cuuint64_t)d->head_dim;
  box[0] = 64;
  if (token_inner) {
    dims[1] = (cuuint64_t)d->block_size;
    dims[2] = (cuuint64_t)d->num_kv_heads;
    strides[0] = (cuuint64_t)d->stride_token * 2;
    strides[1] = (cuuint64_t)d->stride_head * 2;
    box[1] = kTileTokens;
    box[2] = 1;
  } else {
    dims[1] = (cuuint64_t)d->num_kv_heads;
    dims[2] = (cuuint64_t)d->block_size;
    strides[0] = (cuuint64_t)d->stride_head * 2;
    strides[1] = (cuuint64_t)d->stride_token * 2;
    box[1] = 1;
    box[2] = kTileTokens;
  }
  dims[3] = (cuuint64_t)d->num_pages;
  strides[2] = (cuuint64_t)d->stride_page * 2;
  box[3] = 1;
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SEER_OK : SEER_ERR_UNSUPPORTED;
}

// Prompt-query tensor map over q [B][Lq][Hq][D] (Lq = max_blocks * bs): dims
// (D, head, token, batch); box = 64 dims x 1 head x 64 tokens, 128-byte swizzle.
inline seer_status make_q_map(const uint16_t* q, const seer_dims* d, CUtensorMap* map) {
  auto enc = tensor_map_encoder();
  if (!enc) return SEER_ERR_CUDA;
  const cuuint64_t lq = (cuuint64_t)d->max_blocks * d->block_size;
  const cuuint64_t row = (cuuint64_t)d->head_dim * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d->head_dim, (cuuint64_t)d->num_q_heads, lq,
                              (cuuint64_t)d->batch};
  const cuuint64_t strides[3] = {row, row * d->num_q_heads, row * d->num_q_heads * lq};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)kTileTokens, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(q), dims,
                         strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SEER_OK : SEER_ERR_UNSUPPORTED;
}

inline seer_status check_dims(const seer_dims* d) {
  if (d == nullptr) return SEER_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1 || d->max_blocks < 1 ||
      d->num_pages < 1)
    return SEER_ERR_INVALID_ARG;
  if (d->num_q_heads % d->num_kv_heads != 0) return SEER_ERR_INVALID_ARG;
  if (d->head_dim != kHeadDim) return SEER_ERR_UNSUPPORTED;
  if (d->num_q_heads / d->num_kv_heads > kMaxGroup) return SEER_ERR_UNSUPPORTED;
  if (d->block_size != 64 && d->block_size != 128) return SEER_ERR_UNSUPPORTED;
  if (d->max_blocks > kMaxBlocks) return SEER_ERR_UNSUPPORTED;
  if (d->batch > 65535 || d->num_kv_heads > 65535 || d->num_q_heads > 65535)
    return SEER_ERR_UNSUPPORTED;
  if (d->num_pages > INT_MAX) return SEER_ERR_UNSUPPORTED;
  return SEER_OK;
}

inline seer_status check_pool(const seer_dims* d, const uint16_t* pool) {
  if (pool == nullptr) return SEER_ERR_INVALID_ARG;
  if (d->stride_page < 1 || d->stride_token < 1 || d->stride_head < 1) return SEER_ERR_INVALID_ARG;
  if (!aligned(pool, 16) || d->stride_page % 8 || d->stride_token % 8 || d->stride_head % 8)
    return SEER_ERR_UNSUPPORTED;
  return SEER_OK;
}

#define SEER_TRY(expr)                     \
  do {                                     \
    const seer_status st_ = (expr);        \
    if (st_ != SEER_OK) return st_;        \
  } while (0)

// the CUDA error behind this host thread's last SEER_ERR_CUDA
inline cudaError_t& last_cuda_error() {
  static thread_local cudaError_t e = cudaSuccess;
  return e;
}

#define SEER_CUDA(expr)                   \
  do {                                    \
    const cudaError_t seer_e_ = (expr);   \
    if (seer_e_ != cudaSuccess) {         \
      ::seer::last_cuda_error() = seer_e_;  \
      return SEER_ERR_CUDA;               \
    }                                     \
  } while (0)

}  // namespace seer
