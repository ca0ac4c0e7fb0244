// Sliding-window attention with sinks for a ragged chunk of query tokens over
// the paged bf16 cache, on fifth-generation tensor cores.
//
//   the query at position p sees t <= p with t > p - W or t < sinks:
//   out = sum_t e^{scale q . k_t} v_t / sum_t e^{scale q . k_t},  lse = ln of the sum
//
// One CTA per (2 * floor(128 / G) query tokens of one sequence, KV head). The
// rows of an MMA tile are (token, head of the group), so the G heads share
// every key tile and at most G - 1 of 128 rows stay unused; a TMA box of
// 64 dims x G heads x floor(128 / G) tokens lays q out that way.  Two such
// tiles (256 rows) share each 128-key K / V tile.
//   * warp 0 streams K and V (2 stages of 32 KB each) for the key tiles that a
//     row of the CTA sees: the sinks' tiles, then the window's; blocks that no
//     row sees are not looked up (their pages may be gone);
//   * warp 1, one thread: S_i = Q_i K^T (M 128, N 128, SS), O_i += P_i V (A = P in
//     tensor memory); after P_i V_j it issues S_i for tile j + 1 at once (MMAs
//     of one thread execute in order, so S may overwrite P), and tile 1's MMAs
//     run while tile 0's softmax does and the other way round;
//   * warps 2 and 3 zero the V rows of tokens no row of the CTA sees (a zero weight
//     times a cached NaN would be NaN);
//   * warps 4-7 and 8-11, one row per thread: read S from tensor memory (half 0
//     for its maximum, half 1 kept, half 0 again), exponentiate in the exp2
//     domain, write P as bf16 over S and hand each half over as it is done.
// The softmax reference moves only when a row's maximum grows by more than 2^8
// (O and l are then rescaled); P is rounded to bf16 (2^-8), the sum l is of the
// unrounded weights.  Bound by the exponentials (16 per cycle and SM: a
// 256 x 128 tile takes the 2048 cycles of its MMAs) and the hand-offs around
// them.
#include "cache_ops.cuh"
#include "ragged.cuh"
#include "tcgen05.cuh"

namespace seer {

constexpr int kWPThreads = 384;
constexpr int kWPRows = 128;                  // rows of an MMA tile
constexpr int kWPKeys = 128;                  // keys of a tile
constexpr int kWPHalf = kWPKeys * 128;        // 64 dims x 128 rows bf16: 16 KB
constexpr int kWPTile = 2 * kWPHalf;          // a Q, K or V tile
constexpr int kWPStages = 2;
constexpr size_t kWPData = (size_t)(2 + 2 * kWPStages) * kWPTile;  // 192 KB
constexpr size_t kWPSmem = 1024 + kWPData;
constexpr float kWPSlack = 8.f;
#ifndef WP_POLY
#define WP_POLY 4
#endif
constexpr int kWPPolyEvery = WP_POLY;  // one pair in so many takes the FMA pipe's 2^y
constexpr uint32_t kWPIdescS = tc_idesc_bf16(kWPRows, kWPKeys, 0, 0);
constexpr uint32_t kWPIdescPV = tc_idesc_bf16(kWPRows, kHeadDim, 0, 1);

struct WPBars {
  uint64_t q_full;
  uint64_t k_full[kWPStages], k_empty[kWPStages];
  uint64_t v_full[kWPStages], v_fixed[kWPStages], v_empty[kWPStages];
  uint64_t s_full[2], p_ready[2][2], pv_half[2], pv_done[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int b, tile;
  Seq seq;
};

// D[tmem] (+)= A[tmem] * B[smem]^T: A's rows in TMEM lanes, two bf16 of K per column.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::"
      "cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}

// Packed fp32 pairs.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 2^y of a pair, y <= 8, on the FMA pipe: y = n + f with n its nearest integer,
// 2^f by the degree-5 polynomial of least relative error on [-1/2, 1/2] (Remez
// exchange; 2.3e-7 in fp32), times 2^n.  y below -126 gives 2^-126, NaN gives
// NaN.
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t y2) {
  float a, b;
  unpack2(y2, a, b);
  y2 = pack2(max_nan(a, -126.f), max_nan(b, -126.f));
  const uint64_t magic = pack2(12582912.f, 12582912.f), unmagic = pack2(-12582912.f, -12582912.f);
  const uint64_t t2 = add2(y2, magic);
  const uint64_t f2 = fma2(add2(t2, unmagic), pack2(-1.f, -1.f), y2);
  uint64_t r = pack2(1.3276472454890609e-3f, 1.3276472454890609e-3f);
  r = fma2(r, f2, pack2(9.675540961325169e-3f, 9.675540961325169e-3f));
  r = fma2(r, f2, pack2(5.550713092088699e-2f, 5.550713092088699e-2f));
  r = fma2(r, f2, pack2(2.4022120237350464e-1f, 2.4022120237350464e-1f));
  r = fma2(r, f2, pack2(6.931469440460205e-1f, 6.931469440460205e-1f));
  r = fma2(r, f2, pack2(1.0000001192092896f, 1.0000001192092896f));
  float ta, tb;
  unpack2(t2, ta, tb);
  return mul2(r, pack2(__uint_as_float((__float_as_uint(ta) << 23) + 0x3f800000u),
                       __uint_as_float((__float_as_uint(tb) << 23) + 0x3f800000u)));
}

// The lowest n of 64 bits (n clamped to 0 .. 64).
__device__ __forceinline__ uint64_t below(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// The key tiles of a CTA whose rows lie at positions p_min .. p_max.
struct WPKeysOf {
  int p_min, p_max, window, sinks, L;
  int sink_tiles, first_tile, n;  // tile numbers 0 .. sink_tiles - 1, then first_tile ..

  __device__ __forceinline__ int base(int it) const {
    return (it < sink_tiles ? it : first_tile + (it - sink_tiles)) * kWPKeys;
  }
  // some row sees a token of [t, t + len)
  __device__ __forceinline__ bool any(int t, int len) const {
    return t <= p_max && (t < sinks || t + len - 1 > p_min - window);
  }
  // every token of [t, t + len) is seen by some row
  __device__ __forceinline__ bool covered(int t, int len) const {
    return t + len - 1 <= p_max && (t + len <= sinks || t > p_min - window ||
                                    (t < sinks && sinks > p_min - window));
  }
  __device__ __forceinline__ bool seen(int t) const {
    return t <= p_max && (t < sinks || t > p_min - window);
  }
};

__device__ __forceinline__ WPKeysOf wp_keys(int p_min, int p_max, int window, int sinks, int L) {
  WPKeysOf k;
  k.p_min = p_min;
  k.p_max = p_max;
  k.window = window;
  k.L = L;
  k.sinks = min(sinks, p_max + 1);
  k.sink_tiles = ceil_div_i(k.sinks, kWPKeys);
  k.first_tile = max(k.sink_tiles, max(0, p_min - window + 1) / kWPKeys);
  k.n = k.sink_tiles + max(0, p_max / kWPKeys + 1 - k.first_tile);
  return k;
}

__global__ void __launch_bounds__(kWPThreads, 1)
    window_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const WindowPrefillParams p) {
  extern __shared__ uint8_t wp_raw[];
  uint8_t* data = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(wp_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_s = data;
  uint8_t* k_ring = data + 2 * kWPTile;
  uint8_t* v_ring = k_ring + kWPStages * kWPTile;
  __shared__ WPBars bars;

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int h = (int)blockIdx.x % p.Hkv;
  const int item = (int)blockIdx.x / p.Hkv;
  const int per_cta = 2 * p.ntok;

  // ---- which sequence and which of its token tiles (warp 0); meanwhile
  // tensor memory (warp 1), barriers (warp 2), tensor maps (warp 3)
  __shared__ int stop;
  if (warp == 0) {
    int passed = 0, found_b = -1, found_tile = 0;
    Seq found = {0, 0, 0};
    for (int base = 0; base < p.B && found_b < 0; base += 32) {
      const int b = base + lane;
      Seq s = {0, 0, 0};
      if (b < p.B) s = load_seq(p.cu, p.seqlens, b, p.T, p.max_new, p.max_blocks * p.bs, p.status);
      const int cnt = ceil_div_i(s.n, per_cta);
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
        found_b = base + src;
        found_tile = item - __shfl_sync(0xffffffffu, lo, src);
        found.first = __shfl_sync(0xffffffffu, s.first, src);
        found.n = __shfl_sync(0xffffffffu, s.n, src);
        found.L = __shfl_sync(0xffffffffu, s.L, src);
      }
      passed += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      bars.b = found_b;
      bars.tile = found_tile;
      bars.seq = found;
    }
  } else if (warp == 1) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish_alloc_permit();
  } else if (warp == 2) {
    if (lane == 0) {
      mbar_init(&bars.q_full, 1);
      for (int s = 0; s < kWPStages; ++s) {
        mbar_init(&bars.k_full[s], 1);
        mbar_init(&bars.k_empty[s], 1);
        mbar_init(&bars.v_full[s], 1);
        mbar_init(&bars.v_fixed[s], 2);
        mbar_init(&bars.v_empty[s], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.s_full[i], 1);
        mbar_init(&bars.p_ready[i][0], 4);
        mbar_init(&bars.p_ready[i][1], 4);
        mbar_init(&bars.pv_half[i], 1);
        mbar_init(&bars.pv_done[i], 1);
      }
      mbar_init(&bars.mma_done, 1);
      fence_mbar_init();
    }
  } else if (warp == 3) {
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
      // after a wait has run out somewhere in the grid, later CTAs do no work
      // (each run-out wait costs about a second); one thread decides for all
      stop = p.status != nullptr &&
             (*reinterpret_cast<const volatile int32_t*>(p.status) & SEER_DEV_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  if (bars.b < 0) {  // past the last tile: the whole CTA
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const int b = bars.b;
  const Seq seq = bars.seq;
  const int past = seq.L - seq.n;
  const int t0 = bars.tile * per_cta;                      // first query token of the CTA
  const bool two = t0 + p.ntok < seq.n;                    // the second tile has rows
  const int last = min(t0 + per_cta, seq.n) - 1;           // last query token
  const WPKeysOf keys = wp_keys(past + t0, past + last, p.window, p.sinks, seq.L);
  const int nt = stop ? 0 : keys.n;

  if (warp == 0) {
    // ================================================================ copies
    if (nt > 0 && elect_one()) {
      const uint64_t q_policy = policy_evict_first();
      const uint64_t policy = policy_evict_normal();
      const int tiles = two ? 2 : 1;
      mbar_arrive_expect_tx(&bars.q_full, (uint32_t)(tiles * 2 * p.ntok * p.G * 128));
      for (int i = 0; i < tiles; ++i)
        for (int half = 0; half < 2; ++half)
          tma_load_3d(q_s + i * kWPTile + half * kWPHalf, &tm_q, 64 * half, h * p.G,
                      seq.first + t0 + i * p.ntok, &bars.q_full, q_policy);
      const int nb = ceil_div_i(seq.L, p.bs);
      bool ok = true;
      for (int it = 0; it < nt && ok; ++it) {
        const int s0 = keys.base(it), st = it % kWPStages;
        const uint32_t ph = ((it / kWPStages) & 1) ^ 1;
        // the tile's two 64-token pieces: page (or -1: no row sees it) and offset
        int page[2], off[2], loads = 0;
        for (int e = 0; e < 2; ++e) {
          const int t = s0 + 64 * e, j = t / p.bs;
          page[e] = -1;
          off[e] = t - j * p.bs;
          if (j < nb && keys.any(t, 64)) {
            const int64_t pg = page_of(p.page_table, b, j, p.max_blocks);
            if (pg < 0 || pg >= p.num_pages) flag_status(p.status, SEER_DEV_BAD_PAGE);
            page[e] = pg < 0 || pg >= p.num_pages ? 0 : (int)pg;
            ++loads;
          }
        }
        for (int kv = 0; kv < 2 && ok; ++kv) {
          uint64_t* full = kv ? &bars.v_full[st] : &bars.k_full[st];
          if (!mbar_wait(kv ? &bars.v_empty[st] : &bars.k_empty[st], ph)) {
            ok = false;
            break;
          }
          uint8_t* dst = (kv ? v_ring : k_ring) + st * kWPTile;
          mbar_arrive_expect_tx(full, (uint32_t)(loads * kWPTile / 2));
          for (int e = 0; e < 2; ++e) {
            if (page[e] < 0) continue;
            const int c1 = p.token_inner ? off[e] : h, c2 = p.token_inner ? h : off[e];
            for (int half = 0; half < 2; ++half)
              tma_load_4d(dst + half * kWPHalf + e * (kWPHalf / 2), kv ? &tm_v : &tm_k, 64 * half,
                          c1, c2, page[e], full, policy);
          }
        }
      }
      if (!ok) flag_status(p.status, SEER_DEV_TIMEOUT);
      // this CTA's copies land before it retires: the MMA thread consumed all
      // but the newest of each stage, which is waited for here
      for (int it = max(0, nt - kWPStages); it < nt && ok; ++it) {
        const uint32_t ph = (it / kWPStages) & 1;
        if (!mbar_wait(&bars.k_full[it % kWPStages], ph) ||
            !mbar_wait(&bars.v_full[it % kWPStages], ph))
          flag_status(p.status, SEER_DEV_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    // ================================================================ MMA
    if (nt > 0 && elect_one()) {
      bool ok = mbar_wait(&bars.q_full, 0);
      const uint32_t q_addr = smem_u32(q_s), k_addr = smem_u32(k_ring), v_addr = smem_u32(v_ring);
      const int tiles = two ? 2 : 1;
      auto kdesc = [](uint32_t a) { return tc_desc_sw128(a, 16, 1024); };
      auto issue_s = [&](int i, int it) {
        const uint32_t qa = q_addr + i * kWPTile, ka = k_addr + (it % kWPStages) * kWPTile;
#pragma unroll
        for (int k8 = 0; k8 < 8; ++k8) {
          const uint32_t off = (k8 >> 2) * kWPHalf + 32 * (k8 & 3);
          tc_mma_f16_ss(tmem + 128 * i, kdesc(qa + off), kdesc(ka + off), kWPIdescS,
                        k8 > 0 ? 1u : 0u);
        }
        tc_commit(&bars.s_full[i]);
        if (i == tiles - 1) tc_commit(&bars.k_empty[it % kWPStages]);
      };
      auto wait_k = [&](int it) {
        return mbar_wait(&bars.k_full[it % kWPStages], (it / kWPStages) & 1);
      };
      ok = ok && wait_k(0);
      tc_fence_after();
      for (int i = 0; i < tiles && ok; ++i) issue_s(i, 0);
      for (int it = 0; it < nt && ok; ++it) {
        const int st = it % kWPStages;
        const uint32_t ph = (it / kWPStages) & 1;
        ok = mbar_wait(&bars.v_full[st], ph) && mbar_wait(&bars.v_fixed[st], ph);
        for (int i = 0; i < tiles && ok; ++i) {
          // keys 64..127 first, as the softmax hands them over
#pragma unroll
          for (int half = 1; half >= 0; --half) {
            if (!ok || !mbar_wait(&bars.p_ready[i][half], it & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t va = v_addr + st * kWPTile + half * (kWPHalf / 2);
            const uint32_t pa = tmem + 128 * i + 64 * half;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16_ts(tmem + 256 + 128 * i, pa + 8 * kk,
                            tc_desc_sw128(va + 2048 * kk, kWPHalf, 1024), kWPIdescPV,
                            (it > 0 || half == 0 || kk > 0) ? 1u : 0u);
            if (half == 1) tc_commit(&bars.pv_half[i]);
          }
          if (!ok) break;
          if (it == nt - 1) tc_commit(&bars.pv_done[i]);
          if (i == tiles - 1) tc_commit(&bars.v_empty[st]);
          if (it + 1 < nt) {
            if (i == 0 && !wait_k(it + 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_s(i, it + 1);
          }
        }
      }
      if (!ok) flag_status(p.status, SEER_DEV_TIMEOUT);
      // every MMA this thread issued has finished before TMEM is freed
      tc_commit(&bars.mma_done);
      if (!mbar_wait(&bars.mma_done, 0)) flag_status(p.status, SEER_DEV_TIMEOUT);
    }
  } else if (warp < 4) {
    // ========================================= V rows that no row sees: zero
    // (tokens between the sinks and the first window, and past the last query)
    const int tid = threadIdx.x - 64;
    for (int it = 0; it < nt; ++it) {
      const int s0 = keys.base(it), st = it % kWPStages;
      // every tile is waited for in turn (a parity wait cannot tell a phase
      // from the one two before it)
      const bool ok = mbar_wait(&bars.v_full[st], (it / kWPStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        flag_status(p.status, SEER_DEV_TIMEOUT);
        break;
      }
      if (!keys.covered(s0, kWPKeys)) {
        uint8_t* vd = v_ring + st * kWPTile + (tid & 7) * 16 + ((tid >> 3) & 1) * kWPHalf;
        auto zero = [&](int lo, int hi) {  // 64 threads: 4 rows of 16 pieces at a time
          for (int key = lo + (tid >> 4); key < hi; key += 4)
            *reinterpret_cast<uint4*>(vd + key * 128) = make_uint4(0u, 0u, 0u, 0u);
        };
        zero(max(0, keys.sinks - s0), min(kWPKeys, keys.p_min - p.window + 1 - s0));
        zero(max(0, keys.p_max + 1 - s0), kWPKeys);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&bars.v_fixed[st]);
    }
  } else if (warp >= 4) {
    // ============================================================ softmax
    const int i = (warp >> 2) - 1;              // which tile
    const int r = 32 * (warp & 3) + lane;       // this thread's row
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tmem + lanes + 128 * i, o_addr = tmem + lanes + 256 + 128 * i;
    const int tok = t0 + i * p.ntok + r / p.G;  // query token of the sequence
    const bool live = r < p.ntok * p.G && tok < seq.n;
    const int pos = past + tok;
    // positions of the tile's first and last row
    const int pa = past + t0 + i * p.ntok, pz = min(pa + p.ntok, seq.L) - 1;
    if (i == 0 || two) {
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      for (int it = 0; it < nt; ++it) {
        ok = mbar_wait(&bars.s_full[i], it & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int s0 = keys.base(it);
        // every row of the tile sees the whole key tile
        const bool whole = s0 + kWPKeys - 1 <= pa && (s0 > pz - p.window || s0 + kWPKeys <= p.sinks);
        // this row's keys c of the tile: c < hi and (c >= lo or c < sk)
        const int hi = live ? pos - s0 + 1 : 0, lo = pos - p.window + 1 - s0, sk = p.sinks - s0;
#pragma unroll
        for (int half = 1; half >= 0; --half) {
          uint32_t x[64];
          __syncwarp();
          tmem_ld64(s_addr + 64 * half, x);
          if (!whole) {
            const uint64_t seen = below(hi - 64 * half) & (~below(lo - 64 * half) | below(sk - 64 * half));
            const uint32_t w[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(w[c >> 5] & (1u << (c & 31)))) x[c] = 0xff800000u;
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 2)
            m4[(c >> 1) & 3] = fmaxf(m4[(c >> 1) & 3],
                                     fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
          const bool over = mx > m_ref + kWPSlack;
          if (__any_sync(0xffffffffu, over)) {
            float alpha = 1.f;
            if (over) {
              if (m_ref != -INFINITY) alpha = fast_exp2(m_ref - mx);
              m_ref = mx;
            }
            l *= alpha;
            // O holds the tiles before this one (their P V was issued before
            // this tile's S) and, at half 0, this tile's half 1
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
              if (half == 0) {
                ok = mbar_wait(&bars.pv_half[i], it & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
              }
#pragma unroll 1
              for (int c4 = 0; c4 < 4; ++c4) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(o_addr + 32 * c4, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                __syncwarp();
                tmem_st32(o_addr + 32 * c4, o);
              }
            }
          }
          const float ref = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), ref2 = pack2(-ref, -ref);
          uint64_t sum2[2] = {0, 0};
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint64_t y2 = fma2(pack2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])),
                                     scale2, ref2);
            uint64_t e2;
            if (c % kWPPolyEvery == kWPPolyEvery - 1) {
              e2 = exp2_poly2(y2);
            } else {
              float a, e;
              unpack2(y2, a, e);
              e2 = pack2(fast_exp2(a), fast_exp2(e));
            }
            sum2[c & 1] = add2(sum2[c & 1], e2);
            float a, e;
            unpack2(e2, a, e);
            pk[c] = pack_bf16x2(a, e);
          }
          __syncwarp();
          tmem_st32(s_addr + 64 * half, pk);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_ready[i][half]);
          float a, e;
          unpack2(add2(sum2[0], sum2[1]), a, e);
          l += a + e;
        }
        if (!ok) break;
      }
      if (!ok) flag_status(p.status, SEER_DEV_TIMEOUT);
      // ---- epilogue: the last P V, then normalise, bf16 out, natural-log lse
      bool have = ok && nt > 0;
      if (have) {
        have = mbar_wait(&bars.pv_done[i], 0);
        have = __all_sync(0xffffffffu, have);
        if (!have) flag_status(p.status, SEER_DEV_TIMEOUT);
      }
      tc_fence_after();
      if (have) {
        // rows through shared memory (this tile's q, which no MMA reads any
        // more), so that a row leaves as one 256-byte piece
        const int qh = h * p.G + r % p.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint8_t* stage = q_s + i * kWPTile;
#pragma unroll 1
        for (int c2 = 0; c2 < 2; ++c2) {
          uint32_t o[64];
          __syncwarp();
          tmem_ld64(o_addr + 64 * c2, o);
#pragma unroll
          for (int e8 = 0; e8 < 8; ++e8) {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(o[8 * e8 + 0]) * inv, __uint_as_float(o[8 * e8 + 1]) * inv);
            v.y = pack_bf16x2(__uint_as_float(o[8 * e8 + 2]) * inv, __uint_as_float(o[8 * e8 + 3]) * inv);
            v.z = pack_bf16x2(__uint_as_float(o[8 * e8 + 4]) * inv, __uint_as_float(o[8 * e8 + 5]) * inv);
            v.w = pack_bf16x2(__uint_as_float(o[8 * e8 + 6]) * inv, __uint_as_float(o[8 * e8 + 7]) * inv);
            *reinterpret_cast<uint4*>(stage + r * 256 + (((8 * c2 + e8) ^ (r & 15)) << 4)) = v;
          }
        }
        __syncwarp();
        const int r0 = 32 * (warp & 3) + (lane >> 4), piece = lane & 15;
#pragma unroll 4
        for (int k = 0; k < 16; ++k) {
          const int rr = r0 + 2 * k, tk = rr / p.G, g = rr - tk * p.G;
          const int t = t0 + i * p.ntok + tk;
          if (tk < p.ntok && t < seq.n)
            *reinterpret_cast<uint4*>(p.out + ((int64_t)(seq.first + t) * p.Hq + h * p.G + g) * kHeadDim +
                                      8 * piece) =
                *reinterpret_cast<const uint4*>(stage + rr * 256 + ((piece ^ (rr & 15)) << 4));
        }
        if (live && p.lse != nullptr)
          p.lse[(int64_t)qh * p.T + seq.first + tok] =
              l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

cudaError_t run_window_prefill(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const WindowPrefillParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = ensure_smem_limit(window_prefill_kernel, smem_set);
  if (e != cudaSuccess) return e;
  // token tiles: one more than T / per_cta for each sequence's ragged end, but
  // no more than every sequence at max_new
  const int64_t per_cta = 2 * p.ntok;
  int64_t tiles = p.B * ((p.max_new + per_cta - 1) / per_cta);
  const int64_t by_rows = p.T / per_cta + p.B;
  if (by_rows < tiles) tiles = by_rows;
  if (tiles * p.Hkv > 0x7fffffff) return cudaErrorInvalidConfiguration;
  window_prefill_kernel<<<(unsigned)(tiles * p.Hkv), kWPThreads, kWPSmem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace seer
