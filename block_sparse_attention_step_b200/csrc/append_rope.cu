// Append of a ragged batch's new tokens to the paged KV cache, with the
// position rotation of q and k on the way.
//
// Token i of the n_b new ones of sequence b sits at cache position
// pos = seqlen_b - n_b + i.  The first `rot` dims of a q or k row are turned in
// pairs by the angles of the token's position: (x, y) -> (x c - y s, y c + x s),
// c and s from the caller's fp32 table.  Every product and the sum is rounded
// to fp32 on its own (no fma), so a row has the same bits whichever variant or
// thread turns it.  k goes into the cache, rounded once to the cache's type;
// v goes in as it is (bf16) or rounded once (8 bit); q goes to q_out in bf16.
//
// 8-bit cache: one scale per (page, KV head).  With amax the largest finite
// magnitude among the block's new rows and qmax the largest code (448 / 127):
//   * block without earlier rows (or whose scale is 0): the least power of two
//     >= amax / 448 for e4m3 (dividing by it is exact, so a code carries e4m3's
//     own rounding and nothing else); amax / 127 for int8;
//   * else the scale it has, doubled until amax fits.  Doubling keeps the
//     earlier rows' error bounded however often a block grows: an e4m3 code is
//     only re-rounded where it becomes subnormal, an int8 code gains at most
//     half a step per doubling, and the steps double, so all of them together
//     stay below one step of the last scale.
// A scale of 0 says that every row of the block so far is zero.
//
// Two roles share one grid:
//   * block role, one CTA per (touched block, KV head): the block's new rows of
//     k and v come into shared memory by asynchronous copies, all in flight at
//     once, and stay on the SM between the amax and the rounding, so they are
//     read once; the block's keys as the cache gets them replace the raw ones
//     there, for the pooled key (their mean, summed in the order of
//     block_mean.cuh).  Needed for an 8-bit cache and for pooled keys.
//   * row role, a tile of tokens per CTA: q rows, and k and v rows too when the
//     cache is bf16 and no pooled keys are wanted.
// Eight threads take a row, 16 dims each, as two 16-byte chunks that hold
// whole pairs (chunks i and i + rot/16, or neighbours for interleaved pairs).
// Both are HBM-bound streams (about 3 instructions per element).
#include <cuda_fp16.h>

#include "block_mean.cuh"
#include "cache_ops.cuh"
#include "ragged.cuh"

namespace seer {

constexpr int kRowThreads = 8;      // threads per 128-dim row
constexpr int kRowTileRows = 384;   // rows of a row-role tile, about
constexpr int kMaxTileTokens = 128;

// ------------------------------------------------------------- 8-bit codes
template <int CACHE>
struct Code8;

template <>
struct Code8<SEER_CACHE_E4M3> {
  static constexpr float kMax = 448.f;
  // four values (already divided by the scale) to four codes
  static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float (&x)[4]) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  }
  static __device__ __forceinline__ float fresh_scale(float amax) {
    if (!(amax > 0.f)) return 0.f;
    int e;
    const float m = frexpf(amax, &e);  // amax = m 2^e, m in [0.5, 1)
    // 448 = 0.875 * 2^9
    return fmaxf(ldexpf(1.f, m <= 0.875f ? e - 9 : e - 8), 1.17549435e-38f);
  }
};

template <>
struct Code8<SEER_CACHE_INT8> {
  static constexpr float kMax = 127.f;
  static __device__ __forceinline__ uint32_t code(float x) {
    return (uint32_t)max(-127, min(127, __float2int_rn(x))) & 0xffu;
  }
  static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    return code(a) | (code(b) << 8) | (code(c) << 16) | (code(d) << 24);
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)(int8_t)(w >> (8 * e));
  }
  static __device__ __forceinline__ float fresh_scale(float amax) {
    if (!(amax > 0.f)) return 0.f;
    return fmaxf(__fdiv_rn(amax, 127.f), 1.17549435e-38f);
  }
};

// The block's scale after new rows of largest magnitude amax, and the factor
// 2^-k its earlier codes shrink by (1: they stay as they are).
template <int CACHE>
__device__ __forceinline__ float grown_scale(float old, float amax, bool has_old, float* shrink) {
  *shrink = 1.f;
  if (!has_old) return Code8<CACHE>::fresh_scale(amax);
  if (!(amax > 0.f)) return old;
  if (old == 0.f) {
    *shrink = 0.f;
    return Code8<CACHE>::fresh_scale(amax);
  }
  const float limit = __fmul_rn(Code8<CACHE>::kMax, old);
  if (!(amax > limit)) return old;
  // amax <= limit 2^k, by exponents and fractions (exact)
  int ea, el;
  const float ma = frexpf(amax, &ea), ml = frexpf(limit, &el);
  const int k = ea - el + (ma > ml ? 1 : 0);
  *shrink = ldexpf(1.f, -k);
  return ldexpf(old, k);
}

// ------------------------------------------------------------------- rows
__device__ __forceinline__ Seq load_seq(const AppendParams& p, int b) {
  return load_seq(p.cu, p.seqlens, b, p.T, p.max_new, p.max_blocks * p.bs, p.status);
}

// The two chunks of 8 dims a thread (slot 0..7 of its row) holds, and whether
// they are turned.
struct Slot {
  int c0, c1;
  bool turned0, turned1;  // halves style: both or neither
};

__device__ __forceinline__ Slot slot_of(const AppendParams& p, int i) {
  Slot s;
  const int pairs = p.rot >> 4;  // thread slots whose dims are turned, halves style
  if (p.interleaved) {
    s.c0 = 2 * i;
    s.c1 = 2 * i + 1;
    s.turned0 = 8 * s.c0 < p.rot;
    s.turned1 = 8 * s.c1 < p.rot;
  } else if (i < pairs) {
    s.c0 = i;
    s.c1 = i + pairs;
    s.turned0 = s.turned1 = true;
  } else {
    s.c0 = 2 * i;
    s.c1 = 2 * i + 1;
    s.turned0 = s.turned1 = false;
  }
  return s;
}

__device__ __forceinline__ void widen8(uint4 v, float* x) {
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
  x[4] = __uint_as_float(v.z << 16);
  x[5] = __uint_as_float(v.z & 0xffff0000u);
  x[6] = __uint_as_float(v.w << 16);
  x[7] = __uint_as_float(v.w & 0xffff0000u);
}

__device__ __forceinline__ uint4 round8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// A thread's cosines and sines of one table row: halves style, those of pairs
// (8 c0 + e); interleaved, the four of chunk c0, then the four of chunk c1.
struct Turn {
  float4 c[2], w[2];
};

__device__ __forceinline__ Turn load_turn(const AppendParams& p, const Slot& s, int pos) {
  Turn t;
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* row = p.rope + (int64_t)pos * p.rot;
  const int half = p.rot >> 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    t.c[k] = one;
    t.w[k] = zero;
    if (k ? s.turned1 : s.turned0) {
      const int at = p.interleaved ? 4 * (k ? s.c1 : s.c0) : 8 * s.c0 + 4 * k;
      t.c[k] = __ldg(reinterpret_cast<const float4*>(row + at));
      t.w[k] = __ldg(reinterpret_cast<const float4*>(row + half + at));
    }
  }
  return t;
}

// A thread's 16 values (chunk c0, then c1), turned.
__device__ __forceinline__ void turn16(const AppendParams& p, const Slot& s, const Turn& t,
                                       float (&x)[16]) {
  if (p.interleaved) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k ? s.turned1 : s.turned0) {
        float* y = x + 8 * k;
        turn(y[0], y[1], t.c[k].x, t.w[k].x);
        turn(y[2], y[3], t.c[k].y, t.w[k].y);
        turn(y[4], y[5], t.c[k].z, t.w[k].z);
        turn(y[6], y[7], t.c[k].w, t.w[k].w);
      }
    }
  } else if (s.turned0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      turn(x[4 * k], x[8 + 4 * k], t.c[k].x, t.w[k].x);
      turn(x[4 * k + 1], x[9 + 4 * k], t.c[k].y, t.w[k].y);
      turn(x[4 * k + 2], x[10 + 4 * k], t.c[k].z, t.w[k].z);
      turn(x[4 * k + 3], x[11 + 4 * k], t.c[k].w, t.w[k].w);
    }
  }
}

// The table row of a token: its own position or its place in the cache, kept
// inside the table (and flagged) otherwise.
__device__ __forceinline__ int rope_row(const AppendParams& p, int token, int cache_pos) {
  if (p.rot == 0) return 0;
  int pos = p.positions != nullptr ? __ldg(p.positions + token) : cache_pos;
  if (pos < 0 || pos >= p.max_position) {
    flag_status(p.status, SEER_DEV_BAD_POSITION);
    pos = max(0, min(pos, p.max_position - 1));
  }
  return pos;
}

// --------------------------------------------------------------- row role
struct RowShared {
  int bump[kMaxTileTokens];    // sequences that start at this token of the tile
  int rope[kMaxTileTokens];    // table row, -1: no such token
  int64_t at[kMaxTileTokens];  // element offset of the token's cache row of head 0, -1: none
};

__device__ __forceinline__ void row_role(const AppendParams& p, int tile, RowShared& sh) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int t0 = tile * p.tile_tokens;
  const int ntok = min(p.tile_tokens, p.T - t0);
  // the sequence of every token of the tile: sequences before the first token,
  // plus those that start inside the tile up to the token
  int before = 0;
  if (p.cu != nullptr) {
    for (int i = tid; i < ntok; i += nthr) sh.bump[i] = 0;
    __syncthreads();
    for (int base = 1; base <= p.B; base += nthr) {
      const int i = base + tid;
      const int c = i <= p.B ? __ldg(p.cu + i) : INT32_MAX;
      if (c > t0 && c < t0 + ntok) atomicAdd(&sh.bump[c - t0], 1);
      before += __syncthreads_count(c <= t0);
    }
  }
  for (int i = tid; i < ntok; i += nthr) {
    const int t = t0 + i;
    int b = t;
    if (p.cu != nullptr) {
      b = before;
      for (int k = 1; k <= i; ++k) b += sh.bump[k];
    }
    int row = -1;
    int64_t at = -1;
    if (b < p.B) {
      const Seq s = load_seq(p, b);
      if (s.n > 0 && t >= s.first && t < s.first + s.n) {
        const int pos = s.L - s.n + (t - s.first);
        row = rope_row(p, t, pos);
        if (p.rows_kv) {
          const int64_t page = page_of(p.page_table, b, pos / p.bs, p.max_blocks);
          if (page < 0 || page >= p.num_pages) flag_status(p.status, SEER_DEV_BAD_PAGE);
          else at = page * p.stride_page + (int64_t)(pos % p.bs) * p.stride_token;
        }
      }
    }
    sh.rope[i] = row;
    sh.at[i] = at;
  }
  __syncthreads();
  // A warp takes one token's rows [h0, h1) of q, then k, then v: four rows at a
  // time with the token's cosines and sines in registers, the next four read
  // before these are written.
  const int hq = p.q != nullptr ? p.Hq : 0;
  const int hk = p.rows_kv ? p.Hkv : 0;
  const int warp = tid >> 5, lane = tid & 31;
  const Slot sl = slot_of(p, lane % kRowThreads);
  const bool any_turned = sl.turned0 || sl.turned1;
  for (int unit = warp; unit < ntok * p.segments; unit += nthr >> 5) {
    const int i = unit / p.segments;
    const int h0 = (unit - i * p.segments) * p.segment_rows, h1 = h0 + p.segment_rows;
    if (sh.rope[i] < 0) continue;
    const int64_t t = t0 + i;
    Turn tn;
    if (any_turned) tn = load_turn(p, sl, sh.rope[i]);
    auto rows = [&](const uint16_t* src, uint16_t* dst, int64_t dst_stride, int first, int count,
                    bool turned) {
      // rows first .. first + count - 1 of this kind that lie in [h0, h1)
      const int lo = max(h0 - first, 0), hi = min(h1 - first, count);
      const int g = lane / kRowThreads;
      for (int h = lo + g; h < hi; h += 8) {
        const uint4* s0 = reinterpret_cast<const uint4*>(src + (int64_t)h * kHeadDim);
        const bool more = h + 4 < hi;
        uint4 a[2], b[2];
        a[0] = s0[sl.c0];  // plain loads: q may be turned in place
        b[0] = s0[sl.c1];
        if (more) {
          a[1] = s0[4 * 16 + sl.c0];
          b[1] = s0[4 * 16 + sl.c1];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (u == 1 && !more) break;
          if (turned && any_turned) {
            float x[16];
            widen8(a[u], x);
            widen8(b[u], x + 8);
            turn16(p, sl, tn, x);
            a[u] = round8(x);
            b[u] = round8(x + 8);
          }
          uint4* d = reinterpret_cast<uint4*>(dst + (h + 4 * u) * dst_stride);
          d[sl.c0] = a[u];
          d[sl.c1] = b[u];
        }
      }
    };
    if (h0 < hq)
      rows(p.q + t * p.q_stride, p.q_out + t * p.q_out_stride, kHeadDim, 0, hq, true);
    if (h1 > hq && hk > 0 && sh.at[i] >= 0) {
      rows(p.k + t * p.k_stride, static_cast<uint16_t*>(p.k_pool) + sh.at[i], p.stride_head, hq, hk,
           true);
      rows(p.v + t * p.v_stride, static_cast<uint16_t*>(p.v_pool) + sh.at[i], p.stride_head, hq + hk,
           hk, false);
    }
  }
}

// ------------------------------------------------------------- block role
template <int BS>
struct BlockShared {
  // the block's rows, 16 chunks of 16 bytes each: new rows as they come (bf16),
  // earlier keys as the cache holds them; a new key's chunk is replaced by what
  // the cache gets (8-bit codes in the chunk's first half)
  __align__(16) uint8_t keys[BS * kHeadDim * 2];
  __align__(16) uint8_t values[BS * kHeadDim * 2];
  __align__(16) float part[kPoolWarps * kHeadDim];
  float red[2][BS / 8];  // one per warp
  int scan[BS / 8];
  int b, j;
  Seq seq;
  float scale[2], shrink[2];
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// Item number -> (sequence, touched block); false: past the last one.
template <int BS>
__device__ __forceinline__ bool find_block(const AppendParams& p, int item, BlockShared<BS>& sh) {
  constexpr int kThreads = BS * 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sh.b = -1;
  __syncthreads();
  if (p.max_new == 1) {
    if (tid == 0) {
      const Seq s = load_seq(p, item);
      if (s.n > 0) {
        sh.b = item;
        sh.j = (s.L - 1) / p.bs;
        sh.seq = s;
      }
    }
  } else {
    int passed = 0;  // touched blocks of the sequences before this chunk
    for (int base = 0; base < p.B; base += kThreads) {
      const int b = base + tid;
      Seq s = {0, 0, 0};
      int cnt = 0, j0 = 0;
      if (b < p.B) {
        s = load_seq(p, b);
        if (s.n > 0) {
          j0 = (s.L - s.n) / p.bs;
          cnt = (s.L - 1) / p.bs - j0 + 1;
        }
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      int off = passed, total = passed;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) off += sh.scan[w];
        total += sh.scan[w];
      }
      const int lo = off + incl - cnt;
      if (item >= lo && item < lo + cnt) {
        sh.b = b;
        sh.j = j0 + item - lo;
        sh.seq = s;
      }
      passed = total;
      __syncthreads();
      if (passed > item) break;
    }
  }
  __syncthreads();
  return sh.b >= 0;
}

template <int BS, int CACHE>
__device__ __forceinline__ void block_role(const AppendParams& p, int h, BlockShared<BS>& sh) {
  constexpr bool kBf16 = CACHE == SEER_CACHE_BF16;
  constexpr int kThreads = BS * 4;                      // two rows per group of 8 threads
  constexpr int kGroups = kThreads / kRowThreads;       // BS / 2
  constexpr int kBytes = kBf16 ? 2 : 1;                 // per cached element
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = tid / kRowThreads, i = tid % kRowThreads;
  const Seq s = sh.seq;
  const int b = sh.b, j = sh.j;
  const int past = s.L - s.n;
  const int base = j * BS;                       // cache position of the block's row 0
  const int old_rows = max(0, past - base);      // rows it already holds
  const int end = min(BS, s.L - base);           // one past its last new row
  const int64_t page = page_of(p.page_table, b, j, p.max_blocks);
  if (page < 0 || page >= p.num_pages) {
    if (tid == 0) flag_status(p.status, SEER_DEV_BAD_PAGE);
    return;
  }
  const Slot sl = slot_of(p, i);
  const int64_t pool_at = page * p.stride_page + (int64_t)h * p.stride_head;
  uint8_t* kp = static_cast<uint8_t*>(p.k_pool) + pool_at * kBytes;
  uint8_t* vp = static_cast<uint8_t*>(p.v_pool) + pool_at * kBytes;
  const int64_t row_bytes = p.stride_token * kBytes;

  // rows g and g + kGroups of the block, all reads in flight at once; a thread
  // fetches what it works on itself, so it waits for nobody else
  uint4* keys = reinterpret_cast<uint4*>(sh.keys);
  uint4* vals = reinterpret_cast<uint4*>(sh.values);
  bool live[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + u * kGroups;
    live[u] = r >= old_rows && r < end;
    if (live[u]) {
      const int64_t t = s.first + (base + r - past);
      const uint4* ks = reinterpret_cast<const uint4*>(p.k + t * p.k_stride + (int64_t)h * kHeadDim);
      const uint4* vs = reinterpret_cast<const uint4*>(p.v + t * p.v_stride + (int64_t)h * kHeadDim);
      cp_async16(keys + r * 16 + sl.c0, ks + sl.c0);
      cp_async16(keys + r * 16 + sl.c1, ks + sl.c1);
      cp_async16(vals + r * 16 + sl.c0, vs + sl.c0);
      cp_async16(vals + r * 16 + sl.c1, vs + sl.c1);
    } else if (r < old_rows && p.kbar != nullptr) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int chunk = c ? sl.c1 : sl.c0;
        if constexpr (kBf16) cp_async16(keys + r * 16 + chunk, kp + r * row_bytes + 16 * chunk);
        else cp_async8(keys + r * 16 + chunk, kp + r * row_bytes + 8 * chunk);
      }
    }
  }
  float old_scale = 0.f;
  if constexpr (!kBf16) {
    if (tid < 2 && old_rows > 0) old_scale = (tid == 0 ? p.k_scale : p.v_scale)[page * p.Hkv + h];
  }
  cp_async_wait();

  float x[2][16];  // the new keys, turned
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + u * kGroups;
    if (live[u]) {
      widen8(keys[r * 16 + sl.c0], x[u]);
      widen8(keys[r * 16 + sl.c1], x[u] + 8);
      if (sl.turned0 || sl.turned1)
        turn16(p, sl, load_turn(p, sl, rope_row(p, s.first + (base + r - past), base + r)), x[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[u][e] = 0.f;
    }
  }

  if constexpr (kBf16) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + u * kGroups;
      if (!live[u]) continue;
      const uint4 a = round8(x[u]), c = round8(x[u] + 8);
      uint4* kd = reinterpret_cast<uint4*>(kp + r * row_bytes);
      uint4* vd = reinterpret_cast<uint4*>(vp + r * row_bytes);
      kd[sl.c0] = a;
      kd[sl.c1] = c;
      vd[sl.c0] = vals[r * 16 + sl.c0];
      vd[sl.c1] = vals[r * 16 + sl.c1];
      keys[r * 16 + sl.c0] = a;
      keys[r * 16 + sl.c1] = c;
    }
  } else {
    // largest finite magnitudes of the new rows
    float ak = 0.f, av = 0.f;
    bool fine = true;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!live[u]) continue;
      const int r = g + u * kGroups;
      float y[16];
      widen8(vals[r * 16 + sl.c0], y);
      widen8(vals[r * 16 + sl.c1], y + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = fabsf(x[u][e]), c = fabsf(y[e]);
        if (a < INFINITY) ak = fmaxf(ak, a);
        else fine = false;
        if (c < INFINITY) av = fmaxf(av, c);
        else fine = false;
      }
    }
    if (!fine) flag_status(p.status, SEER_DEV_NONFINITE_KV);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ak = fmaxf(ak, __shfl_xor_sync(0xffffffffu, ak, o));
      av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
    }
    if (lane == 0) {
      sh.red[0][warp] = ak;
      sh.red[1][warp] = av;
    }
    __syncthreads();
    if (tid < 2) {  // thread 0: k, thread 1: v
      float a = 0.f;
      for (int w = 0; w < kThreads / 32; ++w) a = fmaxf(a, sh.red[tid][w]);
      float shrink;
      const float now = grown_scale<CACHE>(old_scale, a, old_rows > 0, &shrink);
      if (old_rows == 0 || now != old_scale)
        (tid == 0 ? p.k_scale : p.v_scale)[page * p.Hkv + h] = now;
      sh.scale[tid] = now;
      sh.shrink[tid] = shrink;
    }
    __syncthreads();
    const float inv_k = sh.scale[0] > 0.f ? __frcp_rn(sh.scale[0]) : 0.f;
    const float inv_v = sh.scale[1] > 0.f ? __frcp_rn(sh.scale[1]) : 0.f;
    const float shrink_k = sh.shrink[0], shrink_v = sh.shrink[1];
    auto code8 = [](const float* y, float f) {
      return make_uint2(
          Code8<CACHE>::pack4(__fmul_rn(y[0], f), __fmul_rn(y[1], f), __fmul_rn(y[2], f),
                              __fmul_rn(y[3], f)),
          Code8<CACHE>::pack4(__fmul_rn(y[4], f), __fmul_rn(y[5], f), __fmul_rn(y[6], f),
                              __fmul_rn(y[7], f)));
    };
    auto recode = [&](uint2 w, float f) {
      float y[8];
      Code8<CACHE>::unpack4(w.x, *reinterpret_cast<float(*)[4]>(y));
      Code8<CACHE>::unpack4(w.y, *reinterpret_cast<float(*)[4]>(y + 4));
      return code8(y, f);
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + u * kGroups;
      uint2* kd = reinterpret_cast<uint2*>(kp + r * row_bytes);
      uint2* vd = reinterpret_cast<uint2*>(vp + r * row_bytes);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int chunk = c ? sl.c1 : sl.c0;
        uint2* held = reinterpret_cast<uint2*>(keys + r * 16 + chunk);
        if (live[u]) {
          float y[8];
          widen8(vals[r * 16 + chunk], y);
          const uint2 ck = code8(x[u] + 8 * c, inv_k);
          kd[chunk] = ck;
          vd[chunk] = code8(y, inv_v);
          *held = ck;
        } else if (r < old_rows) {
          // earlier rows: rounded again where the scale grew
          if (shrink_k != 1.f) {
            const uint2 w = recode(kd[chunk], shrink_k);
            kd[chunk] = w;
            *held = w;
          }
          if (shrink_v != 1.f) vd[chunk] = recode(vd[chunk], shrink_v);
        }
      }
    }
  }

  // ---- pooled key: the mean of the rows as the cache holds them
  if (p.kbar == nullptr) return;
  __syncthreads();
  if (warp < kPoolWarps) {
    float4 a;
    if constexpr (kBf16) {
      a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int t = warp; t < end; t += kPoolWarps) {  // the order of pool_warp_partial
        const uint2 w = reinterpret_cast<const uint2*>(sh.keys)[t * 32 + lane];
        a.x += __uint_as_float(w.x << 16);
        a.y += __uint_as_float(w.x & 0xffff0000u);
        a.z += __uint_as_float(w.y << 16);
        a.w += __uint_as_float(w.y & 0xffff0000u);
      }
    } else {
      const float scale = sh.scale[0];
      a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int t = warp; t < end; t += kPoolWarps) {
        float y[4];
        // dims 4 lane .. 4 lane + 3: half of the codes in the first half of chunk lane / 2
        Code8<CACHE>::unpack4(
            reinterpret_cast<const uint32_t*>(sh.keys)[t * 64 + (lane >> 1) * 4 + (lane & 1)], y);
        a.x = __fadd_rn(a.x, __fmul_rn(y[0], scale));
        a.y = __fadd_rn(a.y, __fmul_rn(y[1], scale));
        a.z = __fadd_rn(a.z, __fmul_rn(y[2], scale));
        a.w = __fadd_rn(a.w, __fmul_rn(y[3], scale));
      }
    }
    *reinterpret_cast<float4*>(sh.part + warp * kHeadDim + 4 * lane) = a;
  }
  __syncthreads();
  if (tid < kHeadDim)
    p.kbar[(((int64_t)b * p.Hkv + h) * p.max_blocks + j) * kHeadDim + tid] =
        pool_finish(sh.part, tid, end);
}

// --------------------------------------------------------------- launches
template <int BS, int CACHE>
__global__ void __launch_bounds__(BS * 4, BS == 64 ? 4 : 2) append_blocks_kernel(const AppendParams p) {
  extern __shared__ __align__(16) uint8_t ap_raw[];
  pdl_wait();
  pdl_launch_dependents();
  const int n_blk = p.items * (p.Hkv / p.heads);
  const int c = (int)blockIdx.x;
  if (c < n_blk) {
    BlockShared<BS>& sh = *reinterpret_cast<BlockShared<BS>*>(ap_raw);
    const int per_block = p.Hkv / p.heads;  // CTAs of one block
    if (!find_block<BS>(p, c / per_block, sh)) return;
    for (int i = 0; i < p.heads; ++i) {
      if (i > 0) __syncthreads();  // the pooled key is read out of shared memory
      block_role<BS, CACHE>(p, (c % per_block) * p.heads + i, sh);
    }
  } else {
    row_role(p, c - n_blk, *reinterpret_cast<RowShared*>(ap_raw));
  }
}

__global__ void __launch_bounds__(256) append_rows_kernel(const AppendParams p) {
  __shared__ RowShared sh;
  pdl_wait();
  pdl_launch_dependents();
  row_role(p, (int)blockIdx.x, sh);
}

template <typename Kernel>
static cudaError_t launch_append(Kernel kern, const AppendParams& p, int64_t grid, int threads,
                                 size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int BS, int CACHE>
static cudaError_t launch_blocks(const AppendParams& p, int64_t grid, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = ensure_smem_limit(append_blocks_kernel<BS, CACHE>, smem_set);
  if (e != cudaSuccess) return e;
  static_assert(sizeof(BlockShared<BS>) >= sizeof(RowShared), "both roles share the memory");
  return launch_append(append_blocks_kernel<BS, CACHE>, p, grid, BS * 4, sizeof(BlockShared<BS>),
                       stream);
}

cudaError_t run_append_rope(AppendParams p, int cache, int num_sms, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  p.rows_kv = cache == SEER_CACHE_BF16 && p.kbar == nullptr;
  const int R = (p.q != nullptr ? p.Hq : 0) + (p.rows_kv ? 2 * p.Hkv : 0);
  int64_t tiles = 0;
  if (R > 0) {
    // a warp's share of a token: all its rows, or a part of them where there
    // are too few tokens to keep the SMs busy; a CTA's tile: some kRowTileRows
    // rows (its start -- sequences, lengths, pages, three dependent loads -- costs
    // as much as some 100 rows: 2 x 16K prompt with 56 rows a token, tiles of
    // 128 / 384 / 1024 rows 194 / 177 / 187 us)
    int64_t seg = (32 * (int64_t)num_sms + p.T - 1) / p.T;
    if (seg > (R + 3) / 4) seg = (R + 3) / 4;
    p.segment_rows = (int)(((R + seg - 1) / seg + 3) / 4 * 4);
    p.segments = (R + p.segment_rows - 1) / p.segment_rows;
    p.tile_tokens = p.segments > 1 ? 8 / p.segments : kRowTileRows / R;
    if (p.tile_tokens < 1) p.tile_tokens = 1;
    if (p.tile_tokens > kMaxTileTokens) p.tile_tokens = kMaxTileTokens;
    tiles = ((int64_t)p.T + p.tile_tokens - 1) / p.tile_tokens;
  }
  if (p.rows_kv) return launch_append(append_rows_kernel, p, tiles, 256, 0, stream);
  // touched blocks: n tokens from any place in a block reach at most
  // (n + bs - 2) / bs + 1 blocks
  const int64_t per_seq = ((int64_t)p.max_new + p.bs - 2) / p.bs + 1;
  int64_t items = p.B * per_seq;
  const int64_t by_rows = (int64_t)p.T / p.bs + 2 * (int64_t)p.B;
  if (p.max_new > 1 && by_rows < items) items = by_rows;
  p.items = (int)items;
  // heads of a block per CTA: as many as leave the SMs' resident CTAs twice
  // over (finding the block and its page are paid once for them)
  p.heads = 1;
  for (int hc = 2; hc <= p.Hkv && items * (p.Hkv / hc) >= 8 * (int64_t)num_sms; ++hc)
    if (p.Hkv % hc == 0) p.heads = hc;
  const int64_t grid = items * (p.Hkv / p.heads) + tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.bs == 64) {
    if (cache == SEER_CACHE_BF16) return launch_blocks<64, SEER_CACHE_BF16>(p, grid, stream);
    if (cache == SEER_CACHE_E4M3) return launch_blocks<64, SEER_CACHE_E4M3>(p, grid, stream);
    return launch_blocks<64, SEER_CACHE_INT8>(p, grid, stream);
  }
  if (cache == SEER_CACHE_BF16) return launch_blocks<128, SEER_CACHE_BF16>(p, grid, stream);
  if (cache == SEER_CACHE_E4M3) return launch_blocks<128, SEER_CACHE_E4M3>(p, grid, stream);
  return launch_blocks<128, SEER_CACHE_INT8>(p, grid, stream);
}

// ------------------------------------------------------------------ table
// Row pos: cos, then sin, of pos * base^(-2 i / rot), i = 0 .. rot/2 - 1, the
// angle in fp64 (an fp32 angle of a far position is off by more than the
// table's own rounding).
__global__ void rope_table_kernel(float* table, int max_position, int rot, double base) {
  const int half = rot >> 1;
  const int64_t n = (int64_t)max_position * half;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t pos = e / half;
    const int i = (int)(e - pos * half);
    double sn, cs;
    sincos((double)pos * pow(base, -2.0 * i / rot), &sn, &cs);
    table[pos * rot + i] = (float)cs;
    table[pos * rot + half + i] = (float)sn;
  }
}

cudaError_t run_rope_table(float* table, int max_position, int rot, double base,
                           cudaStream_t stream) {
  const int64_t n = (int64_t)max_position * (rot / 2);
  const int64_t grid = (n + 255) / 256;
  rope_table_kernel<<<(unsigned)(grid < 4096 ? grid : 4096), 256, 0, stream>>>(table, max_position,
                                                                              rot, base);
  return cudaGetLastError();
}

}  // namespace seer
