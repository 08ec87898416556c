// Device helpers shared by the paged-cache kernels.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace lora {

// The sequence that row t of the batch belongs to: the largest s with
// q_off[s] <= t, found by the whole warp in log32(n_seqs) loads; -1 for rows
// of no sequence.  Sequences without new tokens are skipped by taking the
// largest.
__device__ __forceinline__ int seq_of_row(const int32_t* q_off, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_seqs;  // q_off[lo] <= t assumed; the answer is in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const bool le = i <= hi && q_off[i] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    const int new_lo = lo + n * step;
    const int new_hi = new_lo + step - 1;
    lo = new_lo;
    hi = new_hi < hi ? new_hi : hi;
  }
  return lo < n_seqs && q_off[0] <= t ? lo : -1;
}

}  // namespace lora
