// A ragged batch of new tokens: rows cu[b] .. cu[b+1] - 1 belong to sequence b
// and lie at the end of its seqlen tokens (shared by the rotary append and the
// sliding-window prefill).
#pragma once

#include "seer_common.cuh"

namespace seer {

// True in one lane of a converged warp (elect.sync).  Tensor-core and TMA
// instructions are issued under it: a tcgen05.mma of 128 x 128 x 16 took 180
// cycles under `lane == 0` and 64 under this.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// mbar_wait for kernels whose warps wait most of the time next to others that
// are short of issue slots: try_wait without a suspend-time hint, whose own time
// limit decides how long the warp is held (with mbar_wait's hint a third of the
// instructions that the prefill executed were the waits').  Bounded like
// mbar_wait.
__device__ __forceinline__ bool mbar_hold(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  long long t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (ok) return true;
    const long long now = clock64();
    if (t0 == 0) t0 = now;
    else if (now - t0 > (1ll << 31)) return false;
  }
}

struct Seq {
  int first, n, L;  // rows first .. first + n - 1 are its new tokens
};

// n = 0: nothing to do (an inactive slot, or offsets and lengths that do not
// fit, which are flagged); its L is 0, whatever length the slot holds.
__device__ __forceinline__ Seq load_seq(const int32_t* cu, const int32_t* seqlens, int b, int T,
                                        int max_new, int capacity, int32_t* status) {
  Seq s;
  s.L = __ldg(seqlens + b);
  if (cu != nullptr) {
    s.first = __ldg(cu + b);
    const int end = __ldg(cu + b + 1);
    s.n = end - s.first;
    if (s.first < 0 || end < s.first || end > T || s.n > max_new) {
      flag_status(status, SEER_DEV_BAD_TOKENS);
      s.n = 0;
    }
  } else {
    s.first = b;
    s.n = s.L == 0 ? 0 : 1;
  }
  if (s.n > 0 && (s.L < s.n || s.L > capacity)) {
    flag_status(status, SEER_DEV_BAD_TOKENS);
    s.n = 0;
  }
  if (s.n == 0) s.L = 0;
  return s;
}

}  // namespace seer
