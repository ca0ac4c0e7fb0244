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
// A scale of 0 says that every row of the block so far is zero (rows that hold
// NaN or inf next to nothing but zeros get 2^-60 instead).
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
// Bound by HBM where the cache is bf16: 2 x 16K tokens of 40 + 8 + 8 heads with
// pooled keys (950 MB, q by the row role, k and v by the block role) take 156 us,
// 6.1 TB/s, 0.94 of a plain copy's rate; a kernel for each role took 234.  With
// codes a block's CTA loads, reduces and stores in turn and two of them fill an
// SM, the row role's among them: 8 ragged chunks of up to 2.5K tokens of 32 + 8 + 8
// heads into 128-token pages take 53 us with e4m3 codes and 54 with int8, 4.4 TB/s
// (25 and 26 without q, whose rows would take 27 alone; pages of 64: 50 and 53).
// A single token for each of 64 sequences takes 5.9 us (int8 6.3), all of it launch
// and loads that depend on one another.
#include <cuda_fp16.h>

#include "block_mean.cuh"
#include "cache_ops.cuh"
#include "packed.cuh"
#include "ragged.cuh"

namespace seer {

constexpr int kRowThreads = 8;      // threads per 128-dim row
constexpr int kRowTileRows = 384;   // rows of a row-role tile, about
constexpr int kRowTokens = 16;      // its tokens, a multiple of this (the larger CTA's warps)
constexpr int kMaxTileTokens = 128;

// ------------------------------------------------------------- 8-bit codes
template <int CACHE>
struct Code8;

template <>
struct Code8<SEER_CACHE_E4M3> {
  static constexpr float kMax = 448.f;
  // four values (already divided by the scale) to four codes; odd: some may be
  // NaN or inf
  static __device__ __forceinline__ uint32_t pack4(uint64_t ab, uint64_t cd, bool odd) {
    float a, b, c, d;
    unpack2(ab, a, b);
    unpack2(cd, c, d);
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
  static __device__ __forceinline__ uint32_t pack4(uint64_t ab, uint64_t cd, bool odd) {
    float a, b, c, d;
    if (odd) {
      unpack2(ab, a, b);
      unpack2(cd, c, d);
      return code(a) | (code(b) << 8) | (code(c) << 16) | (code(d) << 24);
    }
    // |x| <= 127 (and a rounding): 1.5 * 2^23 + x rounds x to the nearest integer,
    // ties to even, whose two's complement is the sum's low byte.  Against converting
    // instructions here and in the pooled sums: the chunks of 128-token pages 26.5 us
    // instead of 27.6 without q and 53.9 either way with it, of 64-token pages 52.9
    // instead of 51.9
    const uint64_t magic = pack2(12582912.f, 12582912.f);
    unpack2(add2(ab, magic), a, b);
    unpack2(add2(cd, magic), c, d);
    return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                       __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
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
      float* a = x + 4 * k;
      float* b = x + 8 + 4 * k;
      turn(a[0], b[0], t.c[k].x, t.w[k].x);
      turn(a[1], b[1], t.c[k].y, t.w[k].y);
      turn(a[2], b[2], t.c[k].z, t.w[k].z);
      turn(a[3], b[3], t.c[k].w, t.w[k].w);
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

// Item number -> (sequence, touched block) and that sequence's rows; b < 0: past
// the last one.  Every warp works it out for itself, a sequence per lane.
struct Touched {
  int b, j;
  Seq seq;
};

__device__ __forceinline__ Touched find_block(const AppendParams& p, int item) {
  Touched t = {-1, 0, {0, 0, 0}};
  if (p.max_new == 1) {
    const Seq s = load_seq(p, item);
    if (s.n > 0) {
      t.b = item;
      t.j = (s.L - 1) / p.bs;
      t.seq = s;
    }
    return t;
  }
  const int lane = threadIdx.x & 31;
  int passed = 0;  // touched blocks of the sequences before these 32
  for (int base = 0; base < p.B && t.b < 0; base += 32) {
    const int b = base + lane;
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
    const int lo = passed + incl - cnt;
    const unsigned hit = __ballot_sync(0xffffffffu, item >= lo && item < lo + cnt);
    if (hit) {
      const int src = __ffs(hit) - 1;
      t.b = base + src;
      t.j = __shfl_sync(0xffffffffu, j0 + item - lo, src);
      t.seq.first = __shfl_sync(0xffffffffu, s.first, src);
      t.seq.n = __shfl_sync(0xffffffffu, s.n, src);
      t.seq.L = __shfl_sync(0xffffffffu, s.L, src);
    }
    passed += __shfl_sync(0xffffffffu, incl, 31);
  }
  return t;
}

// The larger magnitude of two bf16 pairs, element by element; a NaN stays one.
__device__ __forceinline__ uint32_t max2_abs(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  return d;
}

// Both maxima over the CTA, in every thread (one barrier).
template <int BS>
__device__ __forceinline__ void block_max(float& ak, float& av, BlockShared<BS>& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ak = max_nan(ak, __shfl_xor_sync(0xffffffffu, ak, o));
    av = max_nan(av, __shfl_xor_sync(0xffffffffu, av, o));
  }
  if (lane == 0) {
    sh.red[0][warp] = ak;
    sh.red[1][warp] = av;
  }
  __syncthreads();
  ak = sh.red[0][0];
  av = sh.red[1][0];
#pragma unroll
  for (int w = 1; w < BS / 8; ++w) {
    ak = max_nan(ak, sh.red[0][w]);
    av = max_nan(av, sh.red[1][w]);
  }
}

template <int BS, int CACHE>
__device__ __forceinline__ void block_role(const AppendParams& p, const Touched& where, int h,
                                           BlockShared<BS>& sh) {
  constexpr bool kBf16 = CACHE == SEER_CACHE_BF16;
  constexpr int kThreads = BS * 4;                      // two rows per group of 8 threads
  constexpr int kGroups = kThreads / kRowThreads;       // BS / 2
  constexpr int kBytes = kBf16 ? 2 : 1;                 // per cached element
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = tid / kRowThreads, i = tid % kRowThreads;
  const Seq s = where.seq;
  const int b = where.b, j = where.j;
  const int past = s.L - s.n;
  const int base = j * BS;                       // cache position of the block's row 0
  const int old_rows = max(0, past - base);      // rows it already holds
  const int end = min(BS, s.L - base);           // one past its last new row
  const Slot sl = slot_of(p, i);

  // rows g and g + kGroups of the block, all reads in flight at once; a thread
  // fetches what it works on itself, so it waits for nobody else
  const int64_t t0 = s.first + (base + g - past);  // token of row g
  const uint4* ks = reinterpret_cast<const uint4*>(p.k + t0 * p.k_stride + h * kHeadDim);
  const uint4* vs = reinterpret_cast<const uint4*>(p.v + t0 * p.v_stride + h * kHeadDim);
  uint4* kh = reinterpret_cast<uint4*>(sh.keys) + g * 16;  // row g here; row g + kGroups: + kNext
  uint4* vh = reinterpret_cast<uint4*>(sh.values) + g * 16;
  constexpr int kNext = kGroups * 16;
  bool live[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + u * kGroups;
    live[u] = r >= old_rows && r < end;
    if (live[u]) {
      const uint4* k = u ? ks + kGroups / 8 * p.k_stride : ks;
      const uint4* v = u ? vs + kGroups / 8 * p.v_stride : vs;
      cp_async16(kh + u * kNext + sl.c0, k + sl.c0);
      cp_async16(kh + u * kNext + sl.c1, k + sl.c1);
      cp_async16(vh + u * kNext + sl.c0, v + sl.c0);
      cp_async16(vh + u * kNext + sl.c1, v + sl.c1);
    }
  }
  const int64_t page = page_of(p.page_table, b, j, p.max_blocks);
  if (page < 0 || page >= p.num_pages) {  // the whole CTA
    if (tid == 0) flag_status(p.status, SEER_DEV_BAD_PAGE);
    cp_async_wait();
    return;
  }
  const int64_t pool_at = page * p.stride_page + (int64_t)h * p.stride_head;
  uint8_t* kp = static_cast<uint8_t*>(p.k_pool) + pool_at * kBytes;
  uint8_t* vp = static_cast<uint8_t*>(p.v_pool) + pool_at * kBytes;
  const int64_t row_bytes = p.stride_token * kBytes;
  float old_k = 0.f, old_v = 0.f;  // the block's scales so far
  if (old_rows > 0) {
    if constexpr (!kBf16) {
      old_k = p.k_scale[page * p.Hkv + h];
      old_v = p.v_scale[page * p.Hkv + h];
    }
    if (p.kbar != nullptr) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = g + u * kGroups;
        if (r >= old_rows) continue;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int chunk = c ? sl.c1 : sl.c0;
          if constexpr (kBf16) cp_async16(kh + u * kNext + chunk, kp + r * row_bytes + 16 * chunk);
          else cp_async8(kh + u * kNext + chunk, kp + r * row_bytes + 8 * chunk);
        }
      }
    }
  }
  int at_row[2] = {0, 0};  // the rotation's table rows, fetched behind the copies
  if (sl.turned0 || sl.turned1) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (live[u]) {
        at_row[u] = rope_row(p, (int)t0 + u * kGroups, base + g + u * kGroups);
        const float* row = p.rope + (int64_t)at_row[u] * p.rot + 4 * (p.interleaved ? sl.c0 : 2 * sl.c0);
        asm volatile("prefetch.global.L1 [%0];" ::"l"(row));
        asm volatile("prefetch.global.L1 [%0];" ::"l"(row + (p.rot >> 1)));
      }
    }
  }
  cp_async_wait();

  float key_scale = 1.f;
  float x[2][16];  // the new keys, turned
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (live[u]) {
      widen8(kh[u * kNext + sl.c0], x[u]);
      widen8(kh[u * kNext + sl.c1], x[u] + 8);
      if (sl.turned0 || sl.turned1)
        turn16(p, sl, load_turn(p, sl, at_row[u]), x[u]);
    }
  }
  uint8_t* kd = kp + g * row_bytes;  // row g of the page
  uint8_t* vd = vp + g * row_bytes;

  if constexpr (kBf16) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!live[u]) continue;
      const uint4 a = round8(x[u]), c = round8(x[u] + 8);
      uint4* ku = reinterpret_cast<uint4*>(kd + u * kGroups * row_bytes);
      uint4* vu = reinterpret_cast<uint4*>(vd + u * kGroups * row_bytes);
      ku[sl.c0] = a;
      ku[sl.c1] = c;
      vu[sl.c0] = vh[u * kNext + sl.c0];
      vu[sl.c1] = vh[u * kNext + sl.c1];
      kh[u * kNext + sl.c0] = a;
      kh[u * kNext + sl.c1] = c;
    }
  } else {
    // largest magnitudes of the new rows (a NaN stays one)
    float ak = 0.f, av = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!live[u]) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) ak = max_nan(ak, fabsf(x[u][e]));
      const uint4 a = vh[u * kNext + sl.c0], c = vh[u * kNext + sl.c1];
      const uint32_t top = max2_abs(max2_abs(max2_abs(a.x, a.y), max2_abs(a.z, a.w)),
                                    max2_abs(max2_abs(c.x, c.y), max2_abs(c.z, c.w)));
      av = max_nan(av, max_nan(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u)));
    }
    block_max<BS>(ak, av, sh);
    const bool odd_k = !(ak < INFINITY), odd_v = !(av < INFINITY);
    if (odd_k || odd_v) {
      // (the whole CTA) some value is not finite: over the finite ones
      if (tid == 0) flag_status(p.status, SEER_DEV_NONFINITE_KV);
      ak = av = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!live[u]) continue;
        float y[16];
        widen8(vh[u * kNext + sl.c0], y);
        widen8(vh[u * kNext + sl.c1], y + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (fabsf(x[u][e]) < INFINITY) ak = fmaxf(ak, fabsf(x[u][e]));
          if (fabsf(y[e]) < INFINITY) av = fmaxf(av, fabsf(y[e]));
        }
      }
      __syncthreads();  // everyone has read the first maxima
      block_max<BS>(ak, av, sh);
      // A scale of 0 would say that all is zero, and hide them
      constexpr float kLeast = Code8<CACHE>::kMax * 8.673617379884035e-19f;  // codes of 2^-60
      if (odd_k && ak == 0.f) ak = kLeast;
      if (odd_v && av == 0.f) av = kLeast;
    }
    // every thread works out both scales (the old ones were read by all before
    // the barrier in block_max)
    float shrink_k, shrink_v;
    const float scale_k = grown_scale<CACHE>(old_k, ak, old_rows > 0, &shrink_k);
    const float scale_v = grown_scale<CACHE>(old_v, av, old_rows > 0, &shrink_v);
    if (tid == 0) {
      if (old_rows == 0 || scale_k != old_k) p.k_scale[page * p.Hkv + h] = scale_k;
      if (old_rows == 0 || scale_v != old_v) p.v_scale[page * p.Hkv + h] = scale_v;
    }
    key_scale = scale_k;
    const float inv_k = scale_k > 0.f ? __frcp_rn(scale_k) : 0.f;
    const float inv_v = scale_v > 0.f ? __frcp_rn(scale_v) : 0.f;
    auto code8 = [](const float* y, float f, bool odd) {
      const uint64_t f2 = pack2(f, f);
      uint64_t z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = mul2(pack2(y[2 * e], y[2 * e + 1]), f2);
      return make_uint2(Code8<CACHE>::pack4(z[0], z[1], odd), Code8<CACHE>::pack4(z[2], z[3], odd));
    };
    auto recode = [&](uint2 w, float f) {
      float y[8];
      Code8<CACHE>::unpack4(w.x, *reinterpret_cast<float(*)[4]>(y));
      Code8<CACHE>::unpack4(w.y, *reinterpret_cast<float(*)[4]>(y + 4));
      return code8(y, f, true);
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint2* ku = reinterpret_cast<uint2*>(kd + u * kGroups * row_bytes);
      uint2* vu = reinterpret_cast<uint2*>(vd + u * kGroups * row_bytes);
      uint2* h0 = reinterpret_cast<uint2*>(kh + u * kNext + sl.c0);
      uint2* h1 = reinterpret_cast<uint2*>(kh + u * kNext + sl.c1);
      if (live[u]) {
        float y[16];
        widen8(vh[u * kNext + sl.c0], y);
        widen8(vh[u * kNext + sl.c1], y + 8);
        const uint2 k0 = code8(x[u], inv_k, odd_k), k1 = code8(x[u] + 8, inv_k, odd_k);
        const uint2 v0 = code8(y, inv_v, odd_v), v1 = code8(y + 8, inv_v, odd_v);
        if (sl.c1 == sl.c0 + 1) {  // neighbouring chunks: 16 codes at once
          *reinterpret_cast<uint4*>(ku + sl.c0) = make_uint4(k0.x, k0.y, k1.x, k1.y);
          *reinterpret_cast<uint4*>(vu + sl.c0) = make_uint4(v0.x, v0.y, v1.x, v1.y);
        } else {
          ku[sl.c0] = k0;
          ku[sl.c1] = k1;
          vu[sl.c0] = v0;
          vu[sl.c1] = v1;
        }
        *h0 = k0;
        *h1 = k1;
      } else if (g + u * kGroups < old_rows) {
        // earlier rows: rounded again where the scale grew
        if (shrink_k != 1.f) {
          *h0 = ku[sl.c0] = recode(ku[sl.c0], shrink_k);
          *h1 = ku[sl.c1] = recode(ku[sl.c1], shrink_k);
        }
        if (shrink_v != 1.f) {
          vu[sl.c0] = recode(vu[sl.c0], shrink_v);
          vu[sl.c1] = recode(vu[sl.c1], shrink_v);
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
      // the scale is applied once, to the sum of codes.  A warp's part, at most 16 rows,
      // is exact (e4m3: multiples of 2^-9 below 2^13), and so is the sum of a block of
      // 64; the parts of 128 rows of e4m3 codes may pass 2^15 and round to fp32
      a = make_float4(0.f, 0.f, 0.f, 0.f);
      // dims 4 lane .. 4 lane + 3: half of the codes in the first half of chunk lane / 2
      const uint32_t* w = reinterpret_cast<const uint32_t*>(sh.keys) + (lane >> 1) * 4 + (lane & 1);
      if constexpr (CACHE == SEER_CACHE_INT8) {
        int n[4] = {0, 0, 0, 0};
        for (int t = warp; t < end; t += kPoolWarps) {
          const int x4 = (int)w[t * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) n[e] = __dp4a(x4, 1 << (8 * e), n[e]);
        }
        a = make_float4((float)n[0], (float)n[1], (float)n[2], (float)n[3]);
      } else {
        for (int t = warp; t < end; t += kPoolWarps) {
          float y[4];
          Code8<CACHE>::unpack4(w[t * 64], y);
          a.x += y[0];
          a.y += y[1];
          a.z += y[2];
          a.w += y[3];
        }
      }
    }
    *reinterpret_cast<float4*>(sh.part + warp * kHeadDim + 4 * lane) = a;
  }
  __syncthreads();
  if (tid < kHeadDim)
    p.kbar[(((int64_t)b * p.Hkv + h) * p.max_blocks + j) * kHeadDim + tid] =
        pool_finish(sh.part, tid, end) * key_scale;
}

// --------------------------------------------------------------- launches
template <int BS, int CACHE>
__global__ void __launch_bounds__(BS * 4, BS == 64 ? 4 : 2) append_blocks_kernel(const AppendParams p) {
  extern __shared__ __align__(16) uint8_t ap_raw[];
  pdl_wait();
  pdl_launch_dependents();
  // the block CTAs, spread evenly over the grid: they wait for loads, barriers and
  // arithmetic in turn while the row CTAs stream (2 x 16K prompt 156 us, all
  // of them first 164, last 160; e4m3 chunks alike)
  const int before = (int)((uint64_t)blockIdx.x * p.block_share >> 32);
  const bool is_block = (int)((uint64_t)(blockIdx.x + 1) * p.block_share >> 32) > before;
  if (is_block) {
    const int c = before;
    BlockShared<BS>& sh = *reinterpret_cast<BlockShared<BS>*>(ap_raw);
    const int per_block = p.Hkv / p.heads;  // CTAs of one block
    const Touched where = find_block(p, c / per_block);
    if (where.b < 0) return;
    for (int i = 0; i < p.heads; ++i) {
      if (i > 0) __syncthreads();  // the head before is done with shared memory
      block_role<BS, CACHE>(p, where, (c % per_block) * p.heads + i, sh);
    }
  } else {
    row_role(p, (int)blockIdx.x - before, *reinterpret_cast<RowShared*>(ap_raw));
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
    // as much as some 100 rows), in whole rounds of its warps: 2 x 16K prompt, tiles
    // of 4 / 8 / 9 / 12 / 16 / 24 tokens of 40 rows 189 / 161 / 178 / 167 / 163 / 168 us
    // (before the roles were spread, see append_blocks_kernel)
    int64_t seg = (32 * (int64_t)num_sms + p.T - 1) / p.T;
    if (seg > (R + 3) / 4) seg = (R + 3) / 4;
    p.segment_rows = (int)(((R + seg - 1) / seg + 3) / 4 * 4);
    p.segments = (R + p.segment_rows - 1) / p.segment_rows;
    p.tile_tokens = p.segments > 1 ? 8 / p.segments
                                     : (kRowTileRows / R + kRowTokens - 1) / kRowTokens * kRowTokens;
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
  // heads of a block per CTA: as many as leave the SMs' resident CTAs twice
  // over (finding the block and its page are paid once for them)
  p.heads = 1;
  for (int hc = 2; hc <= p.Hkv && items * (p.Hkv / hc) >= 8 * (int64_t)num_sms; ++hc)
    if (p.Hkv % hc == 0) p.heads = hc;
  const int64_t grid = items * (p.Hkv / p.heads) + tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // block CTAs before CTA c: c * n / grid, rounded down (the share is rounded up
  // by less than 2^-32, so the last one counts)
  p.block_share = (((uint64_t)(grid - tiles) << 32) + (uint64_t)grid - 1) / (uint64_t)grid;
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
