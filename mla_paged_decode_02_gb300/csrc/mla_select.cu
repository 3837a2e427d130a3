// mla_select.cu — the blocks with the largest scores of each token of a ragged batch.
//
// A token that sees n keys has ceil(n / block) blocks. Chosen are its first keep_first and its latest
// keep_last blocks, then those with the largest scores, ties to the lowest index, top_k in all; they
// are written in ascending order, -1 behind them. NaN counts as -inf, and -inf is chosen last.
//
// A score becomes a 32-bit code that ascends with it (kept blocks above all others), and the top_k-th
// largest code is found bit by bit from the top: a bit is set if top_k codes or more are at least as
// large. As soon as exactly top_k are, those are the choice; if that never happens the last bit leaves the
// code itself, and of the blocks that have it the first ones are taken. Counting needs no memory traffic
// and no atomics, whose cost would depend on how alike the scores are.
//
// Bound by latency: reading the row, then some 20 rounds of counting. Up to 1024 blocks a warp takes a
// token, its codes in registers; beyond that a block of 1024 threads does, where a round takes a barrier.
// 128 tokens x 96 blocks 3.1 us, 16 x 4096 6.8, 2048 x 512 8.7, each call on other inputs (histograms of eight bits in
// shared memory, the first form, on the same inputs: 6.7, 16.0, 20.2, where this one took 3.6, 6.4, 8.2).
#include "mla_index.h"
#include "mla_ptx.cuh"
#include "mla_ragged.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kRowWarps = 4;               // tokens of a block where a warp takes a token
constexpr int kRowThreads = 1024;          // of a block that takes one token

// a code that ascends with the score: kept blocks highest, NaN and -inf lowest, -0 as +0
__device__ __forceinline__ uint32_t rank_code(float x, bool kept) {
  if (kept) return 0xFFFFFFFFu;
  if (!(x > -INFINITY)) return 0u;
  const int i = __float_as_int(x + 0.f);
  return i >= 0 ? (uint32_t)i | 0x80000000u : ~(uint32_t)i;
}

// errors that only the device can see, checked by `threads` threads together
__device__ __forceinline__ void check_ragged(const SelectArgs& a, int limit, int first, int threads) {
  for (int b = first; b < a.B; b += threads) {
    const uint32_t bad = ragged_errors(a.cu_q, a.seq_lens, b, a.T, limit);
    if (bad && a.err) atomicOr(a.err, bad);
  }
}

// blocks of token t, or -1 if it belongs to no sequence
__device__ __forceinline__ int blocks_seen(const SelectArgs& a, int limit, int t, int lane) {
  const int b = sequence_of(a.cu_q, a.B, t, lane);
  if (b < 0) return -1;
  const int L = max(0, min(a.seq_lens[b], limit));
  const int seen = keys_seen(t, a.cu_q[b], a.cu_q[b + 1], L, a.causal);
  return seen / a.block + (seen % a.block != 0);
}

// The threshold: codes at least as large as `code` are chosen, but of those that equal it only the first
// `equal`. count(c) is the number of codes that are at least c.
struct Threshold {
  uint32_t code;
  int equal;
};
template <class Count>
__device__ __forceinline__ Threshold find_threshold(int want, Count&& count) {
  uint32_t v = 0;
  int at_least = 0x7FFFFFFF;               // codes >= v (all, for v = 0)
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = v | 1u << bit;
    const int n = count(c);
    if (n < want) continue;
    v = c;
    at_least = n;
    if (n == want) break;
  }
  if (at_least == want) return {v, want};
  const int above = v == 0xFFFFFFFFu ? 0 : count(v + 1);
  return {v, want - above};
}

}  // namespace

// A warp takes a token; lane l holds the codes of blocks l, l + 32, ...
template <int R>
__global__ void __launch_bounds__(32 * kRowWarps) select_warp_kernel(SelectArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int limit = (int)min((int64_t)a.C * a.block, (int64_t)0x7FFFFFFF);
  griddep_wait();                          // the inputs may be the work before's
  griddep_launch_dependents();
  check_ragged(a, limit, blockIdx.x * 32 * kRowWarps + threadIdx.x, gridDim.x * 32 * kRowWarps);
  if (t >= a.T) return;
  // the row is on its way while the token's length is looked up
  const float* row = a.scores + (int64_t)t * a.stride;
  float x[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = lane + 32 * r;
    x[r] = i < a.C ? row[i] : 0.f;
  }
  const int nb = blocks_seen(a, limit, t, lane);
  if (nb < 0) return;
  int32_t* out = a.out + (int64_t)t * a.K;
  const int want = min(a.K, nb);
  for (int i = want + lane; i < a.K; i += 32) out[i] = -1;
  if (nb <= a.K) {
    for (int i = lane; i < nb; i += 32) out[i] = i;
    return;
  }
  uint32_t code[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = lane + 32 * r;
    code[r] = i < nb ? rank_code(x[r], i < a.keep_first || i >= nb - a.keep_last) : 0u;
  }
  const Threshold th = find_threshold(want, [&](uint32_t c) {
    int n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) n += code[r] >= c ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, n);
  });
  int written = 0, equal = 0;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (32 * r >= nb) break;
    // (blocks past the token's, of code 0, come behind every block of that code)
    const uint32_t same = __ballot_sync(0xffffffffu, code[r] == th.code);
    const bool take = code[r] > th.code || (code[r] == th.code && equal + __popc(same & below) < th.equal);
    const uint32_t all = __ballot_sync(0xffffffffu, take);
    if (take) out[written + __popc(all & below)] = lane + 32 * r;
    written += __popc(all);
    equal += __popc(same);
  }
}

// A block takes a token; thread x holds the codes of blocks x, x + 1024, ... in R registers, or (R = 0)
// reads the row again in each round.
template <int R>
__global__ void __launch_bounds__(kRowThreads) select_block_kernel(SelectArgs a) {
  __shared__ int part[2][32];
  __shared__ int2 tally[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = blockIdx.x;
  const int limit = (int)min((int64_t)a.C * a.block, (int64_t)0x7FFFFFFF);
  griddep_wait();                          // the inputs may be the work before's
  griddep_launch_dependents();
  check_ragged(a, limit, t * kRowThreads + tid, gridDim.x * kRowThreads);
  const float* row = a.scores + (int64_t)t * a.stride;
  float x[R > 0 ? R : 1];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + kRowThreads * r;
    x[r] = i < a.C ? row[i] : 0.f;
  }
  const int nb = blocks_seen(a, limit, t, lane);
  if (nb < 0) return;
  int32_t* out = a.out + (int64_t)t * a.K;
  const int want = min(a.K, nb);
  for (int i = want + tid; i < a.K; i += kRowThreads) out[i] = -1;
  if (nb <= a.K) {
    for (int i = tid; i < nb; i += kRowThreads) out[i] = i;
    return;
  }
  auto code_of = [&](int i, float v) { return i < nb ? rank_code(v, i < a.keep_first || i >= nb - a.keep_last) : 0u; };
  uint32_t code[R > 0 ? R : 1];
#pragma unroll
  for (int r = 0; r < R; ++r) code[r] = code_of(tid + kRowThreads * r, x[r]);
  int round = 0;
  const Threshold th = find_threshold(want, [&](uint32_t c) {
    int n = 0;
    if (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) n += code[r] >= c ? 1 : 0;
    } else {
#pragma unroll 8
      for (int i = tid; i < nb; i += kRowThreads) n += code_of(i, row[i]) >= c ? 1 : 0;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    // (two buffers: a warp writes the next round's while others still read this one's)
    int* p = part[round++ & 1];
    if (lane == 0) p[warp] = n;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, p[lane]);
  });
  int written = 0, equal = 0;
  const uint32_t below = (1u << lane) - 1u;
  for (int r = 0; kRowThreads * r < nb; ++r) {
    const int i = tid + kRowThreads * r;
    uint32_t c = 0;
    if (R > 0) {
#pragma unroll
      for (int k = 0; k < R; ++k) c = k == r ? code[k] : c;
    } else {
      c = i < nb ? code_of(i, row[i]) : 0u;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, c > th.code);
    const uint32_t same = __ballot_sync(0xffffffffu, c == th.code);
    __syncthreads();
    if (lane == 0) tally[warp] = make_int2(__popc(over), __popc(same));
    __syncthreads();
    const int2 mine = tally[lane];
    const int over_before = __reduce_add_sync(0xffffffffu, lane < warp ? mine.x : 0);
    const int same_before = __reduce_add_sync(0xffffffffu, lane < warp ? mine.y : 0);
    const int over_all = __reduce_add_sync(0xffffffffu, mine.x), same_all = __reduce_add_sync(0xffffffffu, mine.y);
    // the number of equal codes taken before this thread's
    const int rank = equal + same_before + __popc(same & below);
    const int taken = min(rank, th.equal) - min(equal, th.equal);
    if (c > th.code || (c == th.code && rank < th.equal))
      out[written + over_before + __popc(over & below) + taken] = i;
    written += over_all + min(equal + same_all, th.equal) - min(equal, th.equal);
    equal += same_all;
  }
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.C <= 1024) {
    cfg.gridDim = dim3((a.T + kRowWarps - 1) / kRowWarps);
    cfg.blockDim = dim3(32 * kRowWarps);
    return a.C <= 128   ? cudaLaunchKernelEx(&cfg, select_warp_kernel<4>, a)
           : a.C <= 512 ? cudaLaunchKernelEx(&cfg, select_warp_kernel<16>, a)
                        : cudaLaunchKernelEx(&cfg, select_warp_kernel<32>, a);
  }
  cfg.gridDim = dim3(a.T);
  cfg.blockDim = dim3(kRowThreads);
  return a.C <= 4 * kRowThreads    ? cudaLaunchKernelEx(&cfg, select_block_kernel<4>, a)
         : a.C <= 16 * kRowThreads ? cudaLaunchKernelEx(&cfg, select_block_kernel<16>, a)
                                   : cudaLaunchKernelEx(&cfg, select_block_kernel<0>, a);
}

}  // namespace mla
