// mla_ragged.cuh — the tokens of a ragged batch: which sequence a token belongs to and how many
// keys it sees. Sequence b's new tokens are rows cu_q[b] .. cu_q[b + 1], its last positions.
#pragma once
#include <cstdint>
#include "../../include/mla.h"

namespace mla {

// The sequence of token t, or -1 (a row before the first or behind the last sequence). By a whole
// warp: 32 offsets are compared at a time, two rounds for up to 1024 sequences. A batch with one token
// for each sequence needs one look. With offsets that do not ascend the result is some sequence.
__device__ __forceinline__ int sequence_of(const int32_t* cu_q, int B, int t, int lane) {
  if (t < B && cu_q[t] == t && cu_q[t + 1] == t + 1) return t;
  int lo = 0, hi = B;
  for (;;) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, i < hi && cu_q[i] <= t);
    const int n = below == 0xffffffffu ? 32 : __ffs(~below) - 1;   // offsets up to t
    if (n == 0) return -1;                                         // only in the first round
    lo += (n - 1) * step;
    if (step == 1) break;
    hi = min(hi, lo + step);
  }
  return t < cu_q[lo + 1] ? lo : -1;
}

// Keys that token t of the sequence with rows [start, end) and L keys sees.
__device__ __forceinline__ int keys_seen(int t, int start, int end, int L, int causal) {
  const int n = causal ? L - (end - start) + 1 + (t - start) : L;
  return n < 0 ? 0 : (n > L ? L : n);
}

// Error bits of sequence b: offsets that do not ascend within the T rows, a length outside [0, max_len].
__device__ __forceinline__ uint32_t ragged_errors(const int32_t* cu_q, const int32_t* seq_lens, int b, int T, int max_len) {
  const int s = cu_q[b], e = cu_q[b + 1], L = seq_lens[b];
  return (s < 0 || e < s || e > T ? MLA_DEVERR_CU_Q : 0u) | (L < 0 || L > max_len ? MLA_DEVERR_SEQ_LEN : 0u);
}

}  // namespace mla
