// Sliding-window attention with sinks for a ragged chunk of query tokens over
// the paged bf16 cache, on fifth-generation tensor cores.
//
//   the query at position p sees t <= p with t > p - W or t < sinks:
//   out = sum_t e^{scale q . k_t} v_t / sum_t e^{scale q . k_t},  lse = ln of the sum
//
// One CTA per (floor(128 / G) query tokens of one sequence, KV head), two CTAs per
// SM.  The rows of the MMA tile are (token, head of the group), so the G heads
// share every key tile and at most G - 1 of 128 rows stay unused; a TMA box of
// 64 dims x G heads x floor(128 / G) tokens lays q out that way.
//   * warp 0 streams 64-key tiles of K (3 stages) and V (2 stages) for the keys
//     that a row of the CTA sees: the sinks' tiles, then the window's; blocks
//     that no row sees are not looked up (their pages may be gone);
//   * warp 1, one thread: S = Q K^T (M 128, N 64, SS) into two buffers of tensor
//     memory, O += P V (A = P, in tensor memory over its S).  After P V of tile j
//     it issues S of tile j + 2 into the same buffer at once (MMAs of one thread
//     execute in order), so S of tile j + 1 is there when the softmax of tile j
//     ends;
//   * warps 2 and 3 keep what a row does not see out of its sum (a zero weight
//     times a cached NaN would be NaN): they zero the V rows of tokens no row of
//     the CTA sees, and take NaN and inf out of those that only some rows see;
//     the rows that do see them get them back at the end;
//   * warps 4-7, one row per thread: read S from tensor memory, exponentiate in
//     the exp2 domain, write P as bf16 over S.
// The softmax reference moves only when a row's maximum grows by more than 2^8
// (O and l are then rescaled); P is rounded to bf16 (2^-8), the sum l is of the
// unrounded weights.  Two CTAs run out of step, so one's MMAs, the other's
// softmax and either one's start and end overlap.  Bound by the MMAs: at N 64
// reading Q (4 KB) and K (2 KB) of each K step at 128 B per cycle takes 49
// cycles for 32 cycles of products.
// Where there are too few row tiles for the SMs (a short chunk behind a long
// context) the CTAs of a cluster take a part of a tile's keys each and join their
// states (O, maximum, sum in fp32) over distributed shared memory.  8K prompt (40/8 heads, window 2048, 301
// GFLOP): 359 to 367 us in a loop at the power limit, 316 in a burst (952 TFLOP/s);
// ragged chunks of 129 to 2050 tokens (32/8 heads, window 1000): 94 to 105.  N 128 with two Q
// tiles per CTA and one CTA per SM took 364 to 398, and 17 us instead of 10.7 on a
// chunk of 77 tokens.
#include <cooperative_groups.h>

#include "cache_ops.cuh"
#include "packed.cuh"
#include "ragged.cuh"
#include "tcgen05.cuh"

namespace cg = cooperative_groups;

namespace seer {

constexpr int kWPThreads = 256;
constexpr int kWPRows = 128;                  // rows of the MMA tile
constexpr int kWPKeys = 64;                   // keys of a tile
constexpr int kWPBox = kWPKeys * 128;         // 64 dims x 64 keys bf16: 8 KB
constexpr int kWPTile = 2 * kWPBox;           // a K or V tile
constexpr int kWPHalf = kWPRows * 128;        // 64 dims x 128 rows of q: 16 KB
constexpr int kWPKStages = 3, kWPVStages = 2;
constexpr size_t kWPData = 2 * kWPHalf + (size_t)(kWPKStages + kWPVStages) * kWPTile;  // 112 KB
constexpr int kWPCluster = 8;                 // pieces of a tile's keys, at most
constexpr size_t kWPSmem = kWPData + 1024;    // alignment slack, which holds the barriers too
constexpr float kWPSlack = 8.f;
constexpr uint32_t kWPIdescS = tc_idesc_bf16(kWPRows, kWPKeys, 0, 0);
constexpr uint32_t kWPIdescPV = tc_idesc_bf16(kWPRows, kHeadDim, 0, 1);
constexpr uint32_t kWPCols = 256;             // TMEM: S 2 x 64, O 128

struct WPBars {
  uint64_t q_full;
  uint64_t k_full[kWPKStages], k_empty[kWPKStages];
  uint64_t v_full[kWPVStages], v_fixed[kWPVStages], v_empty[kWPVStages];
  uint64_t s_full[2], p_ready[2], pv_done[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int b, tile, stop;
  int done;  // this CTA's part of the outputs is whole
  Seq seq;
  // tokens that some rows see and some do not and whose value row holds a NaN
  // or inf: bit t - p_min (diagonal), 128 + t - (p_min - window + 1) (window's start)
  uint32_t odd[8];
};
static_assert(sizeof(WPBars) <= 256, "the barriers fit into the alignment slack");

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

// The lowest n of 64 bits (n clamped to 0 .. 64).
__device__ __forceinline__ uint64_t below(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// The key tiles of a CTA whose rows lie at positions p_min .. p_max.
struct WPKeysOf {
  int p_min, p_max, window, sinks;
  int sink_tiles, first_tile, n;  // tile numbers 0 .. sink_tiles - 1, then first_tile ..
  int lo;                         // first of them that is this CTA's

  __device__ __forceinline__ int base(int it) const {
    it += lo;
    return (it < sink_tiles ? it : first_tile + (it - sink_tiles)) * kWPKeys;
  }
  // every row sees all of [t, t + len)
  __device__ __forceinline__ bool whole(int t, int len) const {
    return t + len - 1 <= p_min && (t > p_max - window || t + len <= sinks);
  }
};

__device__ __forceinline__ WPKeysOf wp_keys(int p_min, int p_max, int window, int sinks) {
  WPKeysOf k;
  k.p_min = p_min;
  k.p_max = p_max;
  k.window = window;
  k.sinks = min(sinks, p_max + 1);
  k.sink_tiles = ceil_div_i(k.sinks, kWPKeys);
  k.first_tile = max(k.sink_tiles, max(0, p_min - window + 1) / kWPKeys);
  k.n = k.sink_tiles + max(0, p_max / kWPKeys + 1 - k.first_tile);
  k.lo = 0;
  return k;
}

// The top bit of each half of a bf16 pair that is a NaN or inf (exponent all
// ones), and the pair with those taken as zero.
__device__ __forceinline__ uint32_t odd_of(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t drop_odd(uint32_t w) {
  const uint32_t odd = odd_of(w);
  return w & ~((odd & 0x8000u ? 0xffffu : 0u) | (odd & 0x80000000u ? 0xffff0000u : 0u));
}

// Adds the NaN and inf elements that were taken out of the value rows of partly
// seen tokens to the staged bf16 row (swizzled, see the epilogue) of a query
// that sees them.
__device__ __noinline__ void add_odd(const WindowPrefillParams& p, const uint32_t* odd, int p_min,
                                     int b, int h, int pos, uint8_t* row, int swizzle) {
  for (int bit = 0; bit < 256; ++bit) {
    if (!(odd[bit >> 5] & (1u << (bit & 31)))) continue;
    const int t = bit < 128 ? p_min + bit : p_min - p.window + 1 + bit - 128;
    if (t > pos || (t <= pos - p.window && t >= p.sinks)) continue;
    const int j = t / p.bs;
    const int64_t page = page_of(p.page_table, b, j, p.max_blocks);
    if (page < 0 || page >= p.num_pages) continue;
    const uint16_t* v = p.v_pool + page * p.stride_page + (int64_t)(t - j * p.bs) * p.stride_token +
                        (int64_t)h * p.stride_head;
    for (int e = 0; e < kHeadDim; ++e) {
      const uint32_t w = v[e];
      if ((w & 0x7f80u) != 0x7f80u) continue;
      uint16_t* at = reinterpret_cast<uint16_t*>(row + (((e >> 3) ^ swizzle) << 4)) + (e & 7);
      *at = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float((uint32_t)*at << 16) +
                                                     __uint_as_float(w << 16)));
    }
  }
}

// The same for four values (dims 4 * c4 ..) of a split row; odd: every piece's bits.
__device__ __noinline__ float4 add_odd4(const WindowPrefillParams& p, const uint32_t* odd, int p_min,
                                        int b, int h, int pos, int c4, float4 v) {
  for (int bit = 0; bit < 256; ++bit) {
    if (!(odd[bit >> 5] & (1u << (bit & 31)))) continue;
    const int t = bit < 128 ? p_min + bit : p_min - p.window + 1 + bit - 128;
    if (t > pos || (t <= pos - p.window && t >= p.sinks)) continue;
    const int j = t / p.bs;
    const int64_t page = page_of(p.page_table, b, j, p.max_blocks);
    if (page < 0 || page >= p.num_pages) continue;
    const uint2 w = *reinterpret_cast<const uint2*>(p.v_pool + page * p.stride_page +
                                                    (int64_t)(t - j * p.bs) * p.stride_token +
                                                    (int64_t)h * p.stride_head + 4 * c4);
    const uint32_t e[4] = {w.x << 16, w.x & 0xffff0000u, w.y << 16, w.y & 0xffff0000u};
    float* y = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((e[i] & 0x7f800000u) == 0x7f800000u) y[i] += __uint_as_float(e[i]);
  }
  return v;
}

// A split row tile's partial state in a CTA's shared memory: O [128][128] fp32
// (16-byte pieces swizzled by row), then m, l of each row.
constexpr int kWPPartML = kWPRows * kHeadDim * 4;

// C > 1: the C CTAs of a cluster share the tile's rows and take a part of its key
// tiles each; their states are joined over distributed shared memory.
template <int C>
__global__ void __launch_bounds__(kWPThreads, 2)
    window_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ WindowPrefillParams p) {
  extern __shared__ uint8_t wp_raw[];
  // 1024-byte aligned data (the 128-byte swizzle atom); the barriers go into
  // the slack in front when there are 256 bytes of it, else behind the data
  const uintptr_t raw = reinterpret_cast<uintptr_t>(wp_raw);
  uint8_t* data = reinterpret_cast<uint8_t*>((raw + 1023) & ~uintptr_t(1023));
  WPBars& bars = *reinterpret_cast<WPBars*>(
      reinterpret_cast<uintptr_t>(data) - raw >= 256 ? wp_raw : data + kWPData);
  uint8_t* q_s = data;
  uint8_t* k_ring = data + 2 * kWPHalf;
  uint8_t* v_ring = k_ring + kWPKStages * kWPTile;

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int piece = (int)blockIdx.x % C;
  const int h = (int)blockIdx.x / C % p.Hkv;
  int item = (int)blockIdx.x / C / p.Hkv;

  // ---- which sequence and which of its token tiles (warp 0); meanwhile
  // tensor memory (warp 1), barriers (warp 2), tensor maps (warp 3)
  // The successor may start here, ahead of this grid's tensor memory: its CTAs could
  // hold columns that a CTA of this grid still has to get, and wait for this grid
  // to end.  They cannot as long as no more than two CTAs with tensor memory (256
  // columns each, of 512) fit on an SM by their shared memory: 113 KB here, and
  // prefill_attention_kernel, which is of that size too, is launched without the
  // programmatic attribute.  A kernel with more columns or less shared memory has
  // to move this behind tmem_alloc.
  pdl_launch_dependents();
  if (warp == 0) {
    pdl_wait();  // every other read of global memory comes after the barrier below
    // Row tiles that see a whole window first (whatever their order), then those
    // near the start of their sequence, the longest of each first, so that the
    // grid ends with short CTAs (full causal prompts of 2K / 4K tokens, 32/8 heads:
    // 42 / 136 us, in the order of the rows 53 / 149; ragged chunks vary more from
    // run to run, 94 to 105, than with the order).
    int found_b = -1, found_tile = 0;
    Seq found = {0, 0, 0};
    if (p.max_new == 1 && item < p.B) {  // a row tile per sequence
      found = load_seq(p.cu, p.seqlens, item, p.T, 1, p.max_blocks * p.bs, p.status);
      if (found.n > 0) found_b = item;
    }
    for (int near = p.max_new == 1 ? 2 : 0; near < 2 && found_b < 0; ++near) {
      int passed = 0;
      for (int base = 0; base < p.B && found_b < 0; base += 32) {
        const int b = base + lane;
        Seq s = {0, 0, 0};
        if (b < p.B) s = load_seq(p.cu, p.seqlens, b, p.T, p.max_new, p.max_blocks * p.bs, p.status);
        const int all = ceil_div_i(s.n, p.ntok);
        const int at_start = min(all, ceil_div_i(max(0, p.window - (s.L - s.n)), p.ntok));
        const int cnt = near ? at_start : all - at_start;
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
          found_tile = __shfl_sync(
              0xffffffffu, near ? at_start - 1 - (item - lo) : at_start + (item - lo), src);
          found.first = __shfl_sync(0xffffffffu, s.first, src);
          found.n = __shfl_sync(0xffffffffu, s.n, src);
          found.L = __shfl_sync(0xffffffffu, s.L, src);
        }
        passed += __shfl_sync(0xffffffffu, incl, 31);
      }
      item -= passed;
    }
    if (lane == 0) {
      bars.b = found_b;
      bars.tile = found_tile;
      bars.seq = found;
    }
  } else if (warp == 1) {
    tmem_alloc(&bars.tmem_base, kWPCols);
    tmem_relinquish_alloc_permit();
  } else if (warp == 2) {
    if (lane == 0) {
      mbar_init(&bars.q_full, 1);
      for (int s = 0; s < kWPKStages; ++s) {
        mbar_init(&bars.k_full[s], 1);
        mbar_init(&bars.k_empty[s], 1);
      }
      for (int s = 0; s < kWPVStages; ++s) {
        mbar_init(&bars.v_full[s], 1);
        mbar_init(&bars.v_fixed[s], 2);
        mbar_init(&bars.v_empty[s], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.s_full[i], 1);
        // one per S buffer: a warp may be a tile ahead of another, and its
        // arrival must not count for the other's tile
        mbar_init(&bars.p_ready[i], 4);
        mbar_init(&bars.pv_done[i], 1);
      }
      mbar_init(&bars.mma_done, 1);
      for (int i = 0; i < 8; ++i) bars.odd[i] = 0u;
      bars.done = 1;
      fence_mbar_init();
    }
  } else if (warp == 3) {
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
      pdl_wait();
      // after a wait has run out somewhere in the grid, later CTAs do no work
      // (each run-out wait costs about a second); one thread decides for all
      bars.stop = p.status != nullptr &&
                  (*reinterpret_cast<const volatile int32_t*>(p.status) & SEER_DEV_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  if (bars.b < 0) {  // past the last tile: the whole CTA
    if (warp == 1) tmem_dealloc(tmem, kWPCols);
    return;
  }
  const int b = bars.b;
  const Seq seq = bars.seq;
  const int past = seq.L - seq.n;
  const int t0 = bars.tile * p.ntok;                       // first query token of the CTA
  const int last = min(t0 + p.ntok, seq.n) - 1;            // last query token
  const int pa = past + t0, pz = past + last;              // their positions
  WPKeysOf keys = wp_keys(pa, pz, p.window, p.sinks);
  int nt = bars.stop ? 0 : keys.n;
  if constexpr (C > 1) {
    keys.lo = (int)((int64_t)piece * nt / C);
    nt = (int)((int64_t)(piece + 1) * nt / C) - keys.lo;
  }

  if (warp == 0) {
    // ================================================================ copies
    if (nt > 0 && elect_one()) {
      const uint64_t q_policy = policy_evict_first();
      const uint64_t policy = policy_evict_normal();
      mbar_arrive_expect_tx(&bars.q_full, (uint32_t)(2 * p.ntok * p.G * 128));
      for (int half = 0; half < 2; ++half)
        tma_load_3d(q_s + half * kWPHalf, &tm_q, 64 * half, h * p.G, seq.first + t0, &bars.q_full,
                    q_policy);
      bool ok = true;
      for (int it = 0; it < nt && ok; ++it) {
        const int s0 = keys.base(it), j = s0 / p.bs, off = s0 - j * p.bs;
        int64_t page = page_of(p.page_table, b, j, p.max_blocks);
        if (page < 0 || page >= p.num_pages) {
          flag_status(p.status, SEER_DEV_BAD_PAGE);
          page = 0;  // the copy stays inside the pool, the result is flagged
        }
        const int c1 = p.token_inner ? off : h, c2 = p.token_inner ? h : off;
        const int ks = it % kWPKStages, vs = it % kWPVStages;
        if (!mbar_hold(&bars.k_empty[ks], ((it / kWPKStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&bars.k_full[ks], kWPTile);
        uint8_t* kd = k_ring + ks * kWPTile;
        tma_load_4d(kd, &tm_k, 0, c1, c2, (int)page, &bars.k_full[ks], policy);
        tma_load_4d(kd + kWPBox, &tm_k, 64, c1, c2, (int)page, &bars.k_full[ks], policy);
        if (!mbar_hold(&bars.v_empty[vs], ((it / kWPVStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&bars.v_full[vs], kWPTile);
        uint8_t* vd = v_ring + vs * kWPTile;
        tma_load_4d(vd, &tm_v, 0, c1, c2, (int)page, &bars.v_full[vs], policy);
        tma_load_4d(vd + kWPBox, &tm_v, 64, c1, c2, (int)page, &bars.v_full[vs], policy);
      }
      if (!ok) flag_status(p.status, SEER_DEV_TIMEOUT);
      // this CTA's copies land before it retires: the newest of each stage
      // (older ones were consumed before their stage was used again)
      if (ok) {
        for (int it = max(0, nt - kWPKStages); it < nt; ++it)
          if (!mbar_hold(&bars.k_full[it % kWPKStages], (it / kWPKStages) & 1))
            flag_status(p.status, SEER_DEV_TIMEOUT);
        for (int it = max(0, nt - kWPVStages); it < nt; ++it)
          if (!mbar_hold(&bars.v_full[it % kWPVStages], (it / kWPVStages) & 1))
            flag_status(p.status, SEER_DEV_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    // ================================================================ MMA
    if (nt > 0 && elect_one()) {
      bool ok = mbar_hold(&bars.q_full, 0);
      const uint32_t q_addr = smem_u32(q_s), k_addr = smem_u32(k_ring), v_addr = smem_u32(v_ring);
      auto kdesc = [](uint32_t a) { return tc_desc_sw128(a, 16, 1024); };
      auto issue_s = [&](int it) -> bool {
        const int ks = it % kWPKStages;
        if (!mbar_hold(&bars.k_full[ks], (it / kWPKStages) & 1)) return false;
        tc_fence_after();
        const uint32_t ka = k_addr + ks * kWPTile;
#pragma unroll
        for (int k8 = 0; k8 < 8; ++k8)
          tc_mma_f16_ss(tmem + kWPKeys * (it & 1), kdesc(q_addr + (k8 >> 2) * kWPHalf + 32 * (k8 & 3)),
                        kdesc(ka + (k8 >> 2) * kWPBox + 32 * (k8 & 3)), kWPIdescS, k8 > 0 ? 1u : 0u);
        tc_commit(&bars.s_full[it & 1]);
        tc_commit(&bars.k_empty[ks]);
        return true;
      };
      ok = ok && issue_s(0);
      if (ok && nt > 1) ok = issue_s(1);
      for (int it = 0; it < nt && ok; ++it) {
        const int vs = it % kWPVStages;
        if (!mbar_hold(&bars.v_fixed[vs], (it / kWPVStages) & 1) ||
            !mbar_hold(&bars.p_ready[it & 1], (it >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t va = v_addr + vs * kWPTile, pa_t = tmem + kWPKeys * (it & 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_f16_ts(tmem + 2 * kWPKeys, pa_t + 8 * kk, tc_desc_sw128(va + 2048 * kk, kWPBox, 1024),
                        kWPIdescPV, (it > 0 || kk > 0) ? 1u : 0u);
        tc_commit(&bars.pv_done[it & 1]);
        tc_commit(&bars.v_empty[vs]);
        if (it + 2 < nt) ok = issue_s(it + 2);
      }
      if (!ok) flag_status(p.status, SEER_DEV_TIMEOUT);
      // every MMA this thread issued has finished before TMEM is freed
      tc_commit(&bars.mma_done);
      if (!mbar_hold(&bars.mma_done, 0)) flag_status(p.status, SEER_DEV_TIMEOUT);
    }
  } else if (warp < 4) {
    // ========================================= V rows that no row sees: zero
    // (tokens between the sinks and the first window, and past the last query)
    const int tid = threadIdx.x - 64;
    for (int it = 0; it < nt; ++it) {
      const int s0 = keys.base(it), vs = it % kWPVStages;
      // every tile is waited for in turn (a parity wait cannot tell a phase
      // from the one two before it)
      const bool ok = mbar_hold(&bars.v_full[vs], (it / kWPVStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        flag_status(p.status, SEER_DEV_TIMEOUT);
        break;
      }
      if (!keys.whole(s0, kWPKeys)) {
        // 64 threads: 4 rows of 16 pieces at a time
        uint8_t* vd = v_ring + vs * kWPTile + (tid & 7) * 16 + ((tid >> 3) & 1) * kWPBox;
        // A token that only some rows see weighs zero in the others, and zero
        // times NaN or inf is NaN: such elements are taken out here and added
        // at the end to the rows that do see the token.
        auto take_out = [&](int lo, int hi, int first_bit) {  // keys [lo, hi) of the tile
          for (int k0 = lo + (tid >> 4); k0 < hi; k0 += 16) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              v[u] = k0 + 4 * u < hi ? *reinterpret_cast<const uint4*>(vd + (k0 + 4 * u) * 128)
                                     : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if ((odd_of(v[u].x) | odd_of(v[u].y) | odd_of(v[u].z) | odd_of(v[u].w)) == 0u) continue;
              const int key = k0 + 4 * u, bit = first_bit + key;
              *reinterpret_cast<uint4*>(vd + key * 128) =
                  make_uint4(drop_odd(v[u].x), drop_odd(v[u].y), drop_odd(v[u].z), drop_odd(v[u].w));
              atomicOr(&bars.odd[bit >> 5], 1u << (bit & 31));
            }
          }
        };
        // behind the window's start of some rows (and no sink), ahead of some rows
        const int w0 = pa - p.window + 1;
        take_out(max(0, max(keys.sinks, w0) - s0), min(kWPKeys, min(pz - p.window, pa) + 1 - s0),
                 128 + s0 - w0);
        take_out(max(0, pa + 1 - s0), min(kWPKeys, pz + 1 - s0), s0 - pa);
        auto zero = [&](int lo, int hi) {
          for (int key = lo + (tid >> 4); key < hi; key += 4)
            *reinterpret_cast<uint4*>(vd + key * 128) = make_uint4(0u, 0u, 0u, 0u);
        };
        zero(max(0, keys.sinks - s0), min(kWPKeys, keys.p_min - p.window + 1 - s0));
        zero(max(0, keys.p_max + 1 - s0), kWPKeys);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&bars.v_fixed[vs]);
    }
  } else {
    // ============================================================ softmax
    const int quarter = warp & 3;               // TMEM lanes 32 * quarter ..
    const int r = 32 * quarter + lane;          // this thread's row
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t o_addr = lanes + 2 * kWPKeys;
    const int tok = t0 + r / p.G;               // query token of the sequence
    const bool live = r < p.ntok * p.G && tok < seq.n;
    const int pos = past + tok;
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int it = 0; it < nt; ++it) {
      ok = mbar_hold(&bars.s_full[it & 1], (it >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t s_addr = lanes + kWPKeys * (it & 1);
      uint32_t x[64];
      tmem_ld64(s_addr, x);
      const int s0 = keys.base(it);
      // unless every row sees the whole key tile: this row's keys c, c < hi and
      // (c >= lo or c < sk)
      if (!keys.whole(s0, kWPKeys)) {
        const uint64_t seen = live ? below(pos - s0 + 1) & (~below(pos - p.window + 1 - s0) |
                                                            below(p.sinks - s0))
                                   : 0ull;
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
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          // O is stable once the previous tile's P V is done (the one before it
          // was issued before this tile's S, so the barrier is at most one
          // phase behind)
          ok = mbar_hold(&bars.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
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
        float a, e;
        unpack2(y2, a, e);
        a = fast_exp2(a);  // exp2(-inf) = 0: a key that the row does not see weighs nothing
        e = fast_exp2(e);
        sum2[c & 1] = add2(sum2[c & 1], pack2(a, e));
        pk[c] = pack_bf16x2(a, e);
      }
      __syncwarp();
      tmem_st32(s_addr, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_ready[it & 1]);
      float a, e;
      unpack2(add2(sum2[0], sum2[1]), a, e);
      l += a + e;
    }
    if (!ok) flag_status(p.status, SEER_DEV_TIMEOUT);
    // ---- epilogue: the last P V, then normalise, bf16 out, natural-log lse
    bool have = ok && nt > 0;
    if (have) {
      have = mbar_hold(&bars.pv_done[(nt - 1) & 1], ((nt - 1) >> 1) & 1);
      have = __all_sync(0xffffffffu, have);
      if (!have) flag_status(p.status, SEER_DEV_TIMEOUT);
    }
    tc_fence_after();
    if constexpr (C > 1) {
      // this piece's state; a piece without key tiles adds nothing
      if (bars.stop || (nt > 0 && !have)) {
        bars.done = 0;
      } else {
#pragma unroll 1
        for (int c2 = 0; c2 < 4; ++c2) {
          uint32_t o[32];
          if (nt > 0) {
            __syncwarp();
            tmem_ld32(o_addr + 32 * c2, o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4)
            *reinterpret_cast<uint4*>(data + r * (kHeadDim * 4) + (((8 * c2 + e4) ^ (r & 31)) << 4)) =
                make_uint4(o[4 * e4], o[4 * e4 + 1], o[4 * e4 + 2], o[4 * e4 + 3]);
        }
        *reinterpret_cast<float2*>(data + kWPPartML + 8 * r) = make_float2(m_ref, l);
      }
    } else if (have) {
      // rows through shared memory (q, which no MMA reads any more), so that a
      // row leaves as one 256-byte piece
      const int qh = h * p.G + r % p.G;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint8_t* stage = q_s;
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
      uint32_t odd = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) odd |= bars.odd[i];
      if (odd != 0u && live) add_odd(p, bars.odd, pa, b, h, pos, stage + r * 256, r & 15);
      __syncwarp();
      const int r0 = 32 * quarter + (lane >> 4), piece = lane & 15;
#pragma unroll 4
      for (int k = 0; k < 16; ++k) {
        const int rr = r0 + 2 * k, tk = rr / p.G, g = rr - tk * p.G;
        if (tk < p.ntok && t0 + tk < seq.n)
          *reinterpret_cast<uint4*>(p.out + ((int64_t)(seq.first + t0 + tk) * p.Hq + h * p.G + g) * kHeadDim +
                                    8 * piece) =
              *reinterpret_cast<const uint4*>(stage + rr * 256 + ((piece ^ (rr & 15)) << 4));
      }
      if (live && p.lse != nullptr)
        p.lse[(int64_t)qh * p.T + seq.first + tok] =
            l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kWPCols);
  }
  if constexpr (C > 1) {
    // ---- join: each CTA takes every C-th row, four dims of it a thread
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const uint8_t* part[C];
    int whole = 1;
    uint32_t odd = 0;
#pragma unroll
    for (int q = 0; q < C; ++q) {
      part[q] = cluster.map_shared_rank(data, q);
      const WPBars* at = cluster.map_shared_rank(&bars, q);
      whole &= at->done;
      odd |= at->odd[lane & 7];
    }
    const bool any_odd = __any_sync(0xffffffffu, odd != 0u);
    constexpr int kRows = kWPCluster / C;  // rows whose loads are in flight together
    const int end = whole ? min(p.ntok, seq.n - t0) * p.G : 0;
    for (int r0 = piece + C * kRows * warp; r0 < end; r0 += C * kRows * (kWPThreads / 32)) {
      float2 ml[kRows][C];
      float4 o[kRows][C];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = min(r0 + C * i, kWPRows - 1);
#pragma unroll
        for (int q = 0; q < C; ++q) {
          ml[i][q] = *reinterpret_cast<const float2*>(part[q] + kWPPartML + 8 * r);
          o[i][q] = *reinterpret_cast<const float4*>(part[q] + r * (kHeadDim * 4) +
                                                     ((lane ^ (r & 31)) << 4));
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = r0 + C * i;
        if (r >= end) break;
        const int tk = r / p.G, qh = h * p.G + r - tk * p.G;
        float m = ml[i][0].x;
#pragma unroll
        for (int q = 1; q < C; ++q) m = fmaxf(m, ml[i][q].x);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const float f = fast_exp2(ml[i][q].x - ref);
          l = fmaf(ml[i][q].y, f, l);
          v.x = fmaf(o[i][q].x, f, v.x);
          v.y = fmaf(o[i][q].y, f, v.y);
          v.z = fmaf(o[i][q].z, f, v.z);
          v.w = fmaf(o[i][q].w, f, v.w);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if (any_odd) {
          uint32_t bits[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) bits[k] = __shfl_sync(0xffffffffu, odd, k);
          v = add_odd4(p, bits, pa, b, h, pa + tk, lane, v);
          __syncwarp();
        }
        const int64_t row = seq.first + t0 + tk;
        *reinterpret_cast<uint2*>(p.out + (row * p.Hq + qh) * kHeadDim + 4 * lane) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        if (lane == 0 && p.lse != nullptr)
          p.lse[(int64_t)qh * p.T + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
    // nobody leaves while its state is being read
    cluster.sync();
  }
}

template <int C>
static cudaError_t launch_window_prefill(const CUtensorMap& tq, const CUtensorMap& tk,
                                         const CUtensorMap& tv, const WindowPrefillParams& p,
                                         int64_t rows, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = ensure_smem_limit(window_prefill_kernel<C>, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kWPThreads);
  cfg.dynamicSmemBytes = kWPSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, window_prefill_kernel<C>, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// CTAs per row tile: the C in 1, 2, 4, 8 with the least
//   key tiles of a piece x (1, or 1.3 where SMs hold two CTAs)
//     + for C > 1 a join of 1 + 3 x the share of the 128 rows in use
// (in tiles, 0.65 to 1 us), as long as all CTAs are resident at once with a few
// places to spare for clusters that do not fit a GPC's rest.  Measured, C = 1 / 2 / 4 / 8 (us):
//     1 row tile of 4 rows, 3 key tiles    6.9 /  6.9 /  6.0 /  6.2   rule: 4
//     1 row tile of 4 rows, 65 key tiles  48.0 / 27.6 / 16.7 / 11.6   rule: 8
//     3 row tiles, 7 key tiles            10.7 / 10.9 /  8.9 /  8.4   rule: 8
//    32 row tiles, 17                     20.9 / 17.3 / 14.3 / 14.4   rule: 8
//    35 row tiles, 17                     21.1 / 17.2 / 13.7 / 22.2   rule: 4
//    60 row tiles, 7                      12.2 / 13.0 / 12.9 / 24.0   rule: 4
//    64 row tiles, 33                     38.0 / 26.4 / 19.7 / 32.3   rule: 4
//    74 row tiles, 17                     18.2 / 15.9 / 24.6 / 36.9   rule: 2
//   128 row tiles, 33                     39.5 / 27.4 / 36.5 / 61.8   rule: 2
//   148 row tiles, 17                     18.9 / 19.6 / 38.5 / 64.1   rule: 1
static int pick_pieces(int64_t row_tiles, int64_t keys, int live_rows, int num_sms) {
  const double join = 1.0 + 3.0 * live_rows / kWPRows;
  int best = 1;
  double least = (double)keys;
  for (int c = 2; c <= kWPCluster && row_tiles * c <= 2 * num_sms - 4 * c; c *= 2) {
    const double tile = row_tiles * c <= num_sms ? 1.0 : 1.3;
    const double cost = tile * (double)((keys + c - 1) / c) + join;
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return best;
}

cudaError_t run_window_prefill(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const WindowPrefillParams& p, int num_sms, cudaStream_t stream) {
  // token tiles: T / ntok and one more for each sequence's ragged end, but no
  // more than every sequence at max_new
  int64_t tiles = p.B * (((int64_t)p.max_new + p.ntok - 1) / p.ntok);
  const int64_t by_rows = p.T / p.ntok + p.B;
  if (by_rows < tiles) tiles = by_rows;
  const int64_t rows = tiles * p.Hkv;
  const int ntok = p.ntok < p.max_new ? p.ntok : p.max_new;  // in use
  // key tiles that a row tile can have
  int64_t keys = ((int64_t)p.sinks + kWPKeys - 1) / kWPKeys +
                 ((int64_t)p.window + ntok - 2) / kWPKeys + 2;
  const int64_t most = (int64_t)p.max_blocks * p.bs / kWPKeys;
  if (keys > most) keys = most;
  const int C = pick_pieces(rows, keys, ntok * p.G, num_sms);
  if (rows * C > 0x7fffffff) return cudaErrorInvalidConfiguration;
  switch (C) {
    case 1: return launch_window_prefill<1>(tq, tk, tv, p, rows, stream);
    case 2: return launch_window_prefill<2>(tq, tk, tv, p, rows, stream);
    case 4: return launch_window_prefill<4>(tq, tk, tv, p, rows, stream);
    default: return launch_window_prefill<8>(tq, tk, tv, p, rows, stream);
  }
}

}  // namespace seer
