// A ragged batch of new tokens: rows cu[b] .. cu[b+1] - 1 belong to sequence b
// and lie at the end of its seqlen tokens (shared by the rotary append and the
// sliding-window prefill).
#pragma once

#include "seer_common.cuh"

namespace seer {

// True in one lane of a converged warp.  Code under it is known to run in a
// single thread, so the operands of tensor-core and TMA instructions stay in
// uniform registers; under `lane == 0` the compiler issues each of them through
// a loop over the active lanes (180 cycles per tcgen05.mma instead of the 64
// that a 128 x 128 x 16 one takes).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

struct Seq {
  int first, n, L;  // rows first .. first + n - 1 are its new tokens
};

// n = 0: nothing to do (an inactive slot, or offsets and lengths that do not
// fit, which are flagged).
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
  return s;
}

}  // namespace seer
