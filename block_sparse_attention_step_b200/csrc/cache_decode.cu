// Decode attention (one query token per sequence) over the tokens a block
// list or a sliding window with sinks leaves visible, for a cache in bf16,
// e4m3 or int8.
//
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q . k_t),  lse = ln sum_t w_t
//
// The tokens of one (sequence b, KV head h) row, 64 to a stage, are cut into S
// pieces; up to 8 pieces are the CTAs of one thread-block cluster, which join
// their softmax states over distributed shared memory and write out and lse
// themselves.  Past 8 pieces each cluster writes one partial and the
// log-sum-exp combine follows (whose fp32 weights end at 2^-126).  The order of every sum is fixed by the
// shapes, so results do not change from run to run.
//
// A CTA is four math warps and a copy warp.  The copy warp resolves the
// pieces' blocks and pages (32 stages at a time, one per lane) and streams
// K and V by TMA (128-byte swizzle, evict-first, no multicast) into a ring;
// each math warp owns 16 tokens of every stage.  Tensor-core tile: S^T = K q^T
// with the tokens as M and the group's query heads as N, O^T += V^T P^T with
// the dims as M, so each cached byte serves all G heads from registers.
//
// 8-bit codes become f16 in registers (exact for both types).  Lane (r, c) of
// the K fragment takes 32 neighbouring dims of its token rows with two 16-byte
// loads and uses them as the k indices 2c, 2c+1, 2c+8, 2c+9 of eight MMA
// steps; q is laid out by the same rule, so no transposition is needed.  For V
// it takes 16 neighbouring dims of four tokens, paired byte by byte.  q is
// scaled per head by a power of two that puts its largest element near 2^14
// (a bf16 value then fits f16 exactly unless it is 2^-28 of the largest).
// A block's K scale multiplies its scores.  Its V scale enters the exponent:
// with x_t = log2 w_t, y_t = x_t + log2 vs and a running reference for each,
//   l = sum 2^(x_t - m),   O = sum 2^(y_t - M) code_t,   out = O / l * 2^(M - m),
// so a weight in O is rounded (to f16, 2^-11) relative to the largest contribution
// to O, and l loses nothing, however far the blocks' scales lie apart.  A block of
// scale 0 (all rows zero) has y = -inf: it adds to l alone, its codes are
// taken as zero.
// For a bf16 cache y = x, and P enters as a bf16 hi + lo pair (2^-17).
//
// A reference moves only when a score exceeds it by more than 2^8 (P then stays
// below 256): a vote per tile instead of a maximum over the warp, and no
// rescaling of O or l in between.  Bound by HBM: 256 B (bf16: 512) per token and KV head.
// bf16, 64 sequences x 8 heads, window 4096: 146 us, 6.7 TB/s.  8 bit: 128-byte
// rows 1 KB apart (token-major pages of 8 heads) are what bounds it; the copies
// without the math take 25.3 of 28.3 us (16 x 32K tokens, 10 % of the blocks,
// 109 MB) and 95.6 of 108 us (64 ragged sequences, 485 MB).  The second reference
// and exponential of a token, without which l lost tokens whose V scale is 2^100
// below another's, are 0.8 and 1.5 us of these.  One row of 512 tokens takes
// 5.1 us in 8 pieces: launch, three dependent loads, a copy, the join.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "cache_ops.cuh"
#include "ragged.cuh"

namespace cg = cooperative_groups;

namespace seer {

constexpr int kCDMath = 4;  // math warps
constexpr int kCDThreads = (kCDMath + 1) * 32;
constexpr int kCDCluster = 8;
constexpr int kCDRanked = kRankedBatch;  // sequences ranked by length, at most
constexpr float kCDSlack = 8.f;      // log2 of the largest P

template <int CACHE>
struct CDShape {
  static constexpr bool kBf16 = CACHE == SEER_CACHE_BF16;
  static constexpr int kTileBytes = kTileTokens * kHeadDim * (kBf16 ? 2 : 1);  // K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = kBf16 ? 3 : 4;
  static constexpr int kCtas = kBf16 ? 2 : 3;  // resident per SM (G <= 8)
  static constexpr size_t kRing = (size_t)kStages * kStageBytes;
  static constexpr size_t kSmem = 1024 + kRing;
};

struct __align__(16) CDMeta {
  int base;  // position of the stage's token 0
  float ks;  // K scale
  float lv;  // log2 of the V scale, -inf: 0
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two neighbouring codes (16 bits) to f16x2.
template <int CACHE>
__device__ __forceinline__ uint32_t codes_lo(uint32_t w);
template <int CACHE>
__device__ __forceinline__ uint32_t codes_hi(uint32_t w);

__device__ __forceinline__ uint32_t e4m3x2(uint16_t x) {
  uint32_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
  return y;
}
template <>
__device__ __forceinline__ uint32_t codes_lo<SEER_CACHE_E4M3>(uint32_t w) {
  return e4m3x2((uint16_t)(w & 0xffffu));
}
template <>
__device__ __forceinline__ uint32_t codes_hi<SEER_CACHE_E4M3>(uint32_t w) {
  return e4m3x2((uint16_t)(w >> 16));
}
// int8: f16 bits 0x6400 | u are the number 1024 + u; u = code + 128
__device__ __forceinline__ uint32_t int8x2(uint32_t biased) {
  const uint32_t k = 0x64806480u;  // 1152
  __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&biased),
                      *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t codes_lo<SEER_CACHE_INT8>(uint32_t w) {
  return int8x2(__byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4140));
}
template <>
__device__ __forceinline__ uint32_t codes_hi<SEER_CACHE_INT8>(uint32_t w) {
  return int8x2(__byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4342));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// First stage and stages of a row: the list's blocks, or the sink blocks
// followed by the window's.
struct CDRow {
  int L, nst, sink_blocks, window_block;  // window_block: first block after the sinks' gap
  int a, b;  // token t is visible iff t < a or b <= t < L
};

template <bool WINDOW>
__device__ __forceinline__ CDRow cd_row(const CacheDecodeParams& p, int row, int b) {
  CDRow r;
  r.L = max(0, min(__ldg(p.seqlens + b), p.max_blocks * p.bs));
  const int nsub = p.bs / kTileTokens;
  if constexpr (WINDOW) {
    const int nb = ceil_div_i(r.L, p.bs);
    r.a = min(p.sinks, r.L);
    r.b = max(0, r.L - p.window);  // window <= 2^30
    r.sink_blocks = min(nb, ceil_div_i(r.a, p.bs));
    r.window_block = max(r.sink_blocks, r.b / p.bs);
    r.nst = (r.sink_blocks + max(0, nb - r.window_block)) * nsub;
  } else {
    r.a = r.L;
    r.b = r.L;
    r.sink_blocks = r.window_block = 0;
    r.nst = max(0, min(__ldg(p.n_sel + row), p.k_max)) * nsub;
  }
  return r;
}

template <int CACHE, bool WINDOW, int NT>
__global__ void __launch_bounds__(kCDThreads, NT == 1 ? CDShape<CACHE>::kCtas : 2)
    cache_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const CacheDecodeParams p) {
  using Shape = CDShape<CACHE>;
  constexpr bool kBf16 = Shape::kBf16;
  constexpr int kStages = Shape::kStages;
  extern __shared__ uint8_t cd_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(cd_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t full_bar[kStages], empty_bar[kStages];
  __shared__ CDMeta meta[kStages];
  __shared__ float ml[kCDMath][3][kMaxGroup];  // per warp: M, m, l
  __shared__ float cta_ml[3][kMaxGroup];       // this CTA's M, m, l
  __shared__ __align__(16) int lens[kCDRanked];  // p.by_length
  __shared__ int ranked_b;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G, S = p.S;
  const int place = (int)(blockIdx.x / (unsigned)S);  // of the row in the grid
  const int s = (int)(blockIdx.x % (unsigned)S);
  int b = place / p.Hkv;
  const int h = place - b * p.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_bar[i], 2);  // the copies' arrival and the stage's record
      mbar_init(&empty_bar[i], kCDMath);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  if (!WINDOW && p.by_length) {
    // the b-th longest sequence (of equal ones the first): every thread ranks its own
    const int B4 = (p.B + 3) & ~3;
    for (int i = threadIdx.x; i < B4; i += kCDThreads) lens[i] = i < p.B ? __ldg(p.seqlens + i) : INT_MIN;
    __syncthreads();
    for (int i = threadIdx.x; i < p.B; i += kCDThreads) {
      const int mine = lens[i];
      int rank = 0;
      for (int j = 0; j < B4; j += 4) {
        const int4 o = *reinterpret_cast<const int4*>(lens + j);
        rank += (o.x > mine || (o.x == mine && j < i)) + (o.y > mine || (o.y == mine && j + 1 < i)) +
                (o.z > mine || (o.z == mine && j + 2 < i)) + (o.w > mine || (o.w == mine && j + 3 < i));
      }
      if (rank == b) ranked_b = i;
    }
    __syncthreads();
    b = ranked_b;
  }
  const int row = b * p.Hkv + h;
  const CDRow rw = cd_row<WINDOW>(p, row, b);
  const int lo = (int)((long long)s * rw.nst / S);
  const int n = (int)((long long)(s + 1) * rw.nst / S) - lo;
  const int C = p.C;

  float m[NT][2], my[NT][2], l[NT][2], o[8][NT][4];  // references of l (m) and, 8-bit cache, of O (my)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = my[nt][0] = my[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
  }

  if (warp == kCDMath) {
    // ================================================================ copies
    const uint64_t policy = policy_evict_first();
    const int nsub = p.bs / kTileTokens;
    // Stage t of the piece, one per lane: its block, then its page, then its
    // scales, each a load that depends on the one before.  The next 32 stages
    // go through them while the current 32 are issued.
    auto block_of = [&](int t) {
      const int e = (lo + t) / nsub;
      if constexpr (WINDOW) return e < rw.sink_blocks ? e : rw.window_block + (e - rw.sink_blocks);
      else return __ldg(p.idx + (int64_t)row * p.k_max + e);
    };
    const int nb = ceil_div_i(rw.L, p.bs);
    auto page_at = [&](int t, int j) {  // -1: no such block; bad pages are flagged, page 0 is used
      if (t >= n) return 0;
      if (j < 0 || j >= nb) {
        flag_status(p.status, SEER_DEV_BAD_INDEX);
        return -1;
      }
      const int64_t pg = page_of(p.page_table, b, j, p.max_blocks);
      if (pg >= 0 && pg < p.num_pages) return (int)pg;
      flag_status(p.status, SEER_DEV_BAD_PAGE);
      return 0;
    };
    auto scale_at = [&](const float* scale, int page) {
      return kBf16 || page < 0 ? 1.f : __ldg(scale + (int64_t)page * p.Hkv + h);
    };
    bool ok = true;
    int j = lane < n ? block_of(lane) : 0;
    int page = page_at(lane, j);
    int next_j = 0, next_page = 0;
    float ks = 1.f, vs = 1.f, next_ks = 1.f, next_vs = 1.f;
    for (int base = 0; base < n && ok; base += 32) {
      const int cnt = min(32, n - base);
      const int tok = page < 0 ? 1 << 28  // nothing of this stage is visible
                               : j * p.bs + (lo + base + lane) % nsub * kTileTokens;
      auto issue = [&](int i) {  // stage i of these 32
        const int k = base + i, slot = k % kStages;
        const int pg = max(0, __shfl_sync(0xffffffffu, page, i));
        const int sub = (lo + k) % nsub;
        if (elect_one()) {
          uint8_t* kd = ring + slot * Shape::kStageBytes;
          uint8_t* vd = kd + Shape::kTileBytes;
          const int t0 = sub * kTileTokens;
          const int c1 = p.token_inner ? t0 : h, c2 = p.token_inner ? h : t0;
          mbar_arrive_expect_tx(&full_bar[slot], Shape::kStageBytes);
          if constexpr (kBf16) {
            constexpr int kHalf = Shape::kTileBytes / 2;
            tma_load_4d(kd, &tm_k, 0, c1, c2, pg, &full_bar[slot], policy);
            tma_load_4d(kd + kHalf, &tm_k, 64, c1, c2, pg, &full_bar[slot], policy);
            tma_load_4d(vd, &tm_v, 0, c1, c2, pg, &full_bar[slot], policy);
            tma_load_4d(vd + kHalf, &tm_v, 64, c1, c2, pg, &full_bar[slot], policy);
          } else {
            tma_load_4d(kd, &tm_k, 0, c1, c2, pg, &full_bar[slot], policy);
            tma_load_4d(vd, &tm_v, 0, c1, c2, pg, &full_bar[slot], policy);
          }
        }
        __syncwarp();
      };
      const int t_next = base + 32 + lane;
      if (base + 32 < n) next_j = t_next < n ? block_of(t_next) : 0;
      // the ring's first copies go out before the scales are here
      int issued = 0;
      if (base == 0) {
        ks = scale_at(p.k_scale, page);
        vs = scale_at(p.v_scale, page);
        for (; issued < min(cnt, kStages); ++issued) issue(issued);
      }
      const float lv = kBf16 ? 0.f : log2f(vs);
      for (int i = 0; i < cnt; ++i) {
        const int k = base + i, slot = k % kStages;
        if (i >= issued) {
          ok = mbar_hold(&empty_bar[slot], ((k / kStages) & 1) ^ 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            flag_status(p.status, SEER_DEV_TIMEOUT);
            break;
          }
          issue(i);
        }
        CDMeta mt;
        mt.base = __shfl_sync(0xffffffffu, tok, i);
        mt.ks = __shfl_sync(0xffffffffu, ks, i);
        mt.lv = __shfl_sync(0xffffffffu, lv, i);
        if (lane == 0) {
          meta[slot] = mt;
          mbar_arrive(&full_bar[slot]);
        }
        __syncwarp();
        if (base + 32 < n) {
          if (i == 8) next_page = page_at(t_next, next_j);
          if (i == 16) {
            next_ks = scale_at(p.k_scale, next_page);
            next_vs = scale_at(p.v_scale, next_page);
          }
        }
      }
      j = next_j;
      page = next_page;
      ks = next_ks;
      vs = next_vs;
    }
  } else {
    // ================================================================== math
    const int r = lane >> 2, c = lane & 3, mi = lane >> 3;
    // q^T fragments and the scale of each head column's scores
    uint32_t qb[NT][8][2];
    float cs[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + r;
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (g < G) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + ((int64_t)b * p.Hq + (int64_t)h * G + g) * kHeadDim);
        // dims 32c .. 32c+31; bf16: 16c .. 16c+15 and 64+16c ..
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = __ldg(src + (kBf16 ? 2 * c + (i & 1) + 8 * (i >> 1) : 4 * c + i));
      }
      const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
      if constexpr (kBf16) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          qb[nt][k][0] = u[2 * k];
          qb[nt][k][1] = u[2 * k + 1];
        }
        cs[nt][0] = cs[nt][1] = p.scale_log2;
      } else {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)),
                                 fabsf(__uint_as_float(u[k] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top 2^e in [2^14, 2^15)
        int e = 14 + 127 - (int)(__float_as_uint(top) >> 23);
        e = top > 0.f && top < INFINITY ? max(-126, min(126, e)) : 0;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23) * p.scale_log2;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          qb[nt][k >> 1][k & 1] = pack_f16x2(__uint_as_float(u[k] << 16) * up,
                                             __uint_as_float(u[k] & 0xffff0000u) * up);
        cs[nt][0] = __shfl_sync(0xffffffffu, down, (2 * c) * 4);
        cs[nt][1] = __shfl_sync(0xffffffffu, down, (2 * c + 1) * 4);
      }
    }
    bool ok = true;
    for (int k = 0; k < n; ++k) {
      const int slot = k % kStages;
      ok = mbar_hold(&full_bar[slot], (k / kStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        flag_status(p.status, SEER_DEV_TIMEOUT);
        break;
      }
      const CDMeta mt4 = meta[slot];
      const uint32_t kb = smem_u32(ring + slot * Shape::kStageBytes);
      const uint32_t vb = kb + Shape::kTileBytes;

      // ---- S^T = K q^T over this warp's 16 tokens
      float sacc[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int a = 0; a < 2; ++a)
          sacc[nt][a][0] = sacc[nt][a][1] = sacc[nt][a][2] = sacc[nt][a][3] = 0.f;
      uint32_t va[8][4];
      if constexpr (kBf16) {
        constexpr int kHalf = Shape::kTileBytes / 2;
        const int t0 = warp * 16 + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 16-byte chunk: two k steps
          const uint32_t at = kb + (i >> 1) * kHalf + t0 * 128 + (((2 * c + (i & 1)) ^ (r & 7)) << 4);
          const uint4 x = lds128(at), y = lds128(at + 8 * 128);
          const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(sacc[nt][0], a0, qb[nt][2 * i][0], qb[nt][2 * i][1]);
            mma_bf16_16816(sacc[nt][1], a1, qb[nt][2 * i + 1][0], qb[nt][2 * i + 1][1]);
          }
        }
        const int tok = warp * 16 + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          const int chunk = 2 * mt + (mi & 1);
          ldmatrix_x4_trans(vb + (chunk >> 3) * kHalf + tok * 128 + (((chunk & 7) ^ (tok & 7)) << 4),
                            va[mt][0], va[mt][1], va[mt][2], va[mt][3]);
        }
      } else {
        const int t0 = warp * 16 + r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at = kb + t0 * 128 + (((2 * c + i) ^ (r & 7)) << 4);
          const uint4 x4 = lds128(at), y4 = lds128(at + 8 * 128);
          const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t a[4] = {codes_lo<CACHE>(x[q]), codes_lo<CACHE>(y[q]),
                                   codes_hi<CACHE>(x[q]), codes_hi<CACHE>(y[q])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(sacc[nt][q & 1], a, qb[nt][4 * i + q][0], qb[nt][4 * i + q][1]);
          }
        }
      }
      // V codes of tokens 2c, 2c+1, 2c+8, 2c+9, dims 16r .. 16r+15
      uint4 vw[4];
      if constexpr (!kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = warp * 16 + 2 * c + (i & 1) + 8 * (i >> 1);
          vw[i] = lds128(vb + t * 128 + ((r ^ (t & 7)) << 4));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[slot]);

      // ---- tokens the row does not see: no score, no value (a cached NaN
      // times a zero weight would be NaN)
      const int tb = mt4.base + warp * 16;  // position of this warp's first token
      const bool all_seen = (tb + 16 <= rw.a || tb >= rw.b) && tb + 16 <= rw.L;
      bool in0 = true, in1 = true;
      if (!all_seen) {
        auto seen = [&](int t) { return t < rw.a || (t >= rw.b && t < rw.L); };
        in0 = seen(tb + r);
        in1 = seen(tb + r + 8);
        const bool v0 = seen(tb + 2 * c), v1 = seen(tb + 2 * c + 1);
        const bool v2 = seen(tb + 2 * c + 8), v3 = seen(tb + 2 * c + 9);
        if constexpr (kBf16) {
          const uint32_t mlo = (v0 ? 0x0000ffffu : 0u) | (v1 ? 0xffff0000u : 0u);
          const uint32_t mhi = (v2 ? 0x0000ffffu : 0u) | (v3 ? 0xffff0000u : 0u);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            va[mt][0] &= mlo;
            va[mt][1] &= mlo;
            va[mt][2] &= mhi;
            va[mt][3] &= mhi;
          }
        } else {
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
          if (!v0) vw[0] = z;
          if (!v1) vw[1] = z;
          if (!v2) vw[2] = z;
          if (!v3) vw[3] = z;
        }
      }
      if constexpr (!kBf16) {
        if (mt4.lv == -INFINITY) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vw[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }

      // ---- weights relative to the lazily moved references
      float x[NT][4];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // a score past this moves a reference (-inf less -inf, a NaN, leaves m's)
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          top[e] = (kBf16 ? m[nt][e] : fminf(m[nt][e], my[nt][e] - mt4.lv)) + kCDSlack;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = sacc[nt][0][e] + sacc[nt][1][e];
          const bool in = e < 2 ? in0 : in1;
          x[nt][e] = in ? v * (kBf16 ? cs[nt][e & 1] : cs[nt][e & 1] * mt4.ks) : -INFINITY;
          over |= x[nt][e] > top[e & 1];
        }
      }
      // the factor by which what was summed shrinks when a reference moves to
      // the tile's maximum (over the warp's tokens of a head column)
      auto move_to = [](float& ref, float a, float b) {
        float mx = fmaxf(a, b);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float to = fmaxf(ref, mx);
        const float alpha = to == -INFINITY ? 1.f : fast_exp2(ref - to);
        ref = to;
        return alpha;
      };
      auto shrink_o = [&](int nt, int e, float alpha) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          o[mt][nt][e] *= alpha;
          o[mt][nt][2 + e] *= alpha;
        }
      };
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float alpha = move_to(m[nt][e], x[nt][e], x[nt][2 + e]);
            l[nt][e] *= alpha;
            if constexpr (kBf16) shrink_o(nt, e, alpha);
            else shrink_o(nt, e, move_to(my[nt][e], x[nt][e] + mt4.lv, x[nt][2 + e] + mt4.lv));
          }
        }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
          pr[e] = fast_exp2(x[nt][e] - ref);
        }
        l[nt][0] += pr[0] + pr[2];
        l[nt][1] += pr[1] + pr[3];
        if constexpr (kBf16) {
          uint32_t h0, l0, h1, l1;
          split_bf16x2(pr[0], pr[1], h0, l0);
          split_bf16x2(pr[2], pr[3], h1, l1);
          ph[nt][0] = movmatrix_trans(h0);
          ph[nt][1] = movmatrix_trans(h1);
          pl[nt][0] = movmatrix_trans(l0);
          pl[nt][1] = movmatrix_trans(l1);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ref = my[nt][e & 1] == -INFINITY ? 0.f : my[nt][e & 1];
            pr[e] = fast_exp2(x[nt][e] + (mt4.lv - ref));
          }
          ph[nt][0] = movmatrix_trans(pack_f16x2(pr[0], pr[1]));
          ph[nt][1] = movmatrix_trans(pack_f16x2(pr[2], pr[3]));
        }
      }
      // ---- O^T += V^T P^T
      if constexpr (kBf16) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(o[mt][nt], va[mt], ph[nt][0], ph[nt][1]);
            mma_bf16_16816(o[mt][nt], va[mt], pl[nt][0], pl[nt][1]);
          }
        }
      } else {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&vw[0]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&vw[1]);
        const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&vw[2]);
        const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&vw[3]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // dims 16r + 4q .. + 3: tiles 2q and 2q + 1
          const uint32_t p0 = __byte_perm(w0[q], w1[q], 0x5140), p1 = __byte_perm(w0[q], w1[q], 0x7362);
          const uint32_t p2 = __byte_perm(w2[q], w3[q], 0x5140), p3 = __byte_perm(w2[q], w3[q], 0x7362);
          const uint32_t a0[4] = {codes_lo<CACHE>(p0), codes_hi<CACHE>(p0), codes_lo<CACHE>(p2),
                                  codes_hi<CACHE>(p2)};
          const uint32_t a1[4] = {codes_lo<CACHE>(p1), codes_hi<CACHE>(p1), codes_lo<CACHE>(p3),
                                  codes_hi<CACHE>(p3)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(o[2 * q][nt], a0, ph[nt][0], ph[nt][1]);
            mma_f16_16816(o[2 * q + 1][nt], a1, ph[nt][0], ph[nt][1]);
          }
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        l[nt][e] = v;
      }
    }
  }
  // Every copy this CTA started has landed before the ring is used again: the
  // math warps waited for each stage, and so does the copy warp (bounded) in
  // case one of them gave up.
  if (warp == kCDMath && lane == 0) {
    for (int k = max(0, n - kStages); k < n; ++k)
      if (!mbar_hold(&full_bar[k % kStages], (k / kStages) & 1))
        flag_status(p.status, SEER_DEV_TIMEOUT);
  }
  __syncthreads();

  // ---- join the warps' states: [warp][head][dim] in the ring
  float* ow = reinterpret_cast<float*>(ring);
  if (warp < kCDMath) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = nt * 8 + 2 * c + e;
        if (g < G) {
          if (r == 0) {
            ml[warp][0][g] = kBf16 ? m[nt][e] : my[nt][e];
            ml[warp][1][g] = m[nt][e];
            ml[warp][2][g] = l[nt][e];
          }
          float* dst = ow + (size_t)(warp * G + g) * kHeadDim;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            if constexpr (kBf16) {
              dst[mt * 16 + r] = o[mt][nt][e];
              dst[mt * 16 + r + 8] = o[mt][nt][2 + e];
            } else {
              *reinterpret_cast<float2*>(dst + 16 * r + 2 * mt) =
                  make_float2(o[mt][nt][e], o[mt][nt][2 + e]);
            }
          }
        }
      }
    }
  }
  __syncthreads();
  float* co = ow + (size_t)kCDMath * G * kHeadDim;  // the CTA's state [head][dim]
  for (int e = threadIdx.x; e < G * kHeadDim; e += kCDThreads) {
    const int g = e / kHeadDim;
    float M = -INFINITY, m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kCDMath; ++w) {
      M = fmaxf(M, ml[w][0][g]);
      m = fmaxf(m, ml[w][1][g]);
    }
    float L = 0.f, O = 0.f;
    const float ref_o = M == -INFINITY ? 0.f : M, ref_l = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < kCDMath; ++w) {
      O = fmaf(ow[(size_t)w * G * kHeadDim + e], fast_exp2(ml[w][0][g] - ref_o), O);
      L = fmaf(ml[w][2][g], fast_exp2(ml[w][1][g] - ref_l), L);
    }
    co[e] = O;
    if (e % kHeadDim == 0) {
      cta_ml[0][g] = M;
      cta_ml[1][g] = m;
      cta_ml[2][g] = L;
    }
  }
  // ---- join the cluster's CTAs: each takes its part of the outputs
  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) cluster.sync();
  else __syncthreads();
  const int rank = C > 1 ? (int)cluster.block_rank() : 0;
  for (int e = rank * kCDThreads + threadIdx.x; e < G * kHeadDim; e += C * kCDThreads) {
    const int g = e / kHeadDim, d = e - g * kHeadDim;
    float Mq[kCDCluster], mq[kCDCluster], M = -INFINITY, m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kCDCluster; ++q) {
      if (q < C) {
        Mq[q] = C > 1 ? *cluster.map_shared_rank(&cta_ml[0][g], q) : cta_ml[0][g];
        mq[q] = kBf16 ? Mq[q] : C > 1 ? *cluster.map_shared_rank(&cta_ml[1][g], q) : cta_ml[1][g];
        M = fmaxf(M, Mq[q]);
        m = fmaxf(m, mq[q]);
      }
    }
    const float ref_o = M == -INFINITY ? 0.f : M, ref_l = m == -INFINITY ? 0.f : m;
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int q = 0; q < kCDCluster; ++q) {
      if (q < C) {
        L = fmaf(C > 1 ? *cluster.map_shared_rank(&cta_ml[2][g], q) : cta_ml[2][g],
                 fast_exp2(mq[q] - ref_l), L);
        O = fmaf(C > 1 ? *cluster.map_shared_rank(&co[e], q) : co[e], fast_exp2(Mq[q] - ref_o), O);
      }
    }
    float v = L == 0.f ? 0.f : O / L;
    if constexpr (!kBf16) {
      // times 2^(M - m) by halves: the whole may lie below the normal numbers where
      // its product with O / l does not
      const float half = L == 0.f ? 0.f : fast_exp2(0.5f * (M - m));
      v = v * half * half;
    }
    const float lse = L == 0.f ? -INFINITY : (m + log2f(L)) * kLn2;
    const int64_t orow = (int64_t)b * p.Hq + (int64_t)h * G + g;
    if (p.o_part != nullptr) {
      const int64_t part = orow * (S / C) + s / C;
      p.o_part[part * kHeadDim + d] = v;
      if (d == 0) p.lse_part[part] = lse;
    } else {
      p.out[orow * kHeadDim + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
      if (d == 0 && p.lse_out != nullptr) p.lse_out[orow] = lse;
    }
  }
  if (C > 1) cluster.sync();  // nobody leaves while its state is being read
}

template <int CACHE, bool WINDOW, int NT>
static cudaError_t launch_cache_decode(const CUtensorMap& tk, const CUtensorMap& tv,
                                       const CacheDecodeParams& p, cudaStream_t stream) {
  auto kern = cache_decode_kernel<CACHE, WINDOW, NT>;
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * p.S));
  cfg.blockDim = dim3(kCDThreads);
  cfg.dynamicSmemBytes = CDShape<CACHE>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, tk, tv, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t run_cache_decode(const CUtensorMap& tk, const CUtensorMap& tv,
                             const CacheDecodeParams& p, int cache, bool window,
                             cudaStream_t stream) {
  auto by_heads = [&](auto cache_tag, auto window_tag) {
    constexpr int kCache = decltype(cache_tag)::value;
    constexpr bool kWindow = decltype(window_tag)::value;
    return p.G <= 8 ? launch_cache_decode<kCache, kWindow, 1>(tk, tv, p, stream)
                    : launch_cache_decode<kCache, kWindow, 2>(tk, tv, p, stream);
  };
  using E4 = std::integral_constant<int, SEER_CACHE_E4M3>;
  using I8 = std::integral_constant<int, SEER_CACHE_INT8>;
  using BF = std::integral_constant<int, SEER_CACHE_BF16>;
  if (window) {
    if (cache == SEER_CACHE_E4M3) return by_heads(E4{}, std::true_type{});
    if (cache == SEER_CACHE_INT8) return by_heads(I8{}, std::true_type{});
    return by_heads(BF{}, std::true_type{});
  }
  return cache == SEER_CACHE_E4M3 ? by_heads(E4{}, std::false_type{})
                                  : by_heads(I8{}, std::false_type{});
}

}  // namespace seer
