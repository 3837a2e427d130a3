// mla_select.cu — the blocks with the largest scores of each token of a ragged batch.
//
// A token that sees n keys has ceil(n / block) blocks. Chosen are its first keep_first and its latest
// keep_last blocks, then those with the largest scores, ties to the lowest index, top_k in all; they
// are written in ascending order, -1 behind them. NaN counts as -inf, and -inf is chosen last.
#include "mla_index.h"
#include "mla_ragged.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kSelectThreads = 256;

// a code that ascends with the score: kept blocks highest, NaN and -inf lowest, -0 as +0
__device__ __forceinline__ uint32_t rank_code(float x, bool kept) {
  if (kept) return 0xFFFFFFFFu;
  if (!(x > -INFINITY)) return 0u;
  const int i = __float_as_int(x + 0.f);
  return i >= 0 ? (uint32_t)i | 0x80000000u : ~(uint32_t)i;
}

}  // namespace

// A CTA takes one token: a radix selection, eight bits of the threshold at a time, then one pass that
// writes what lies above the threshold and the first of what equals it.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(SelectArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sum[kSelectThreads / 32];
  __shared__ int pick[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x;
  const int limit = (int)min((int64_t)a.C * a.block, (int64_t)0x7FFFFFFF);
  for (int b = t * kSelectThreads + threadIdx.x; b < a.B; b += gridDim.x * kSelectThreads) {
    const uint32_t bad = ragged_errors(a.cu_q, a.seq_lens, b, a.T, limit);
    if (bad && a.err) atomicOr(a.err, bad);
  }
  const int b = sequence_of(a.cu_q, a.B, t, lane);
  if (b < 0) return;
  const int L = max(0, min(a.seq_lens[b], limit));
  const int seen = keys_seen(t, a.cu_q[b], a.cu_q[b + 1], L, a.causal);
  const int nb = seen / a.block + (seen % a.block != 0);
  int32_t* out = a.out + (int64_t)t * a.K;
  const float* row = a.scores + (int64_t)t * a.stride;
  const int want = min(a.K, nb);
  for (int i = want + threadIdx.x; i < a.K; i += kSelectThreads) out[i] = -1;
  if (nb <= a.K) {
    for (int i = threadIdx.x; i < nb; i += kSelectThreads) out[i] = i;
    return;
  }
  auto code = [&](int i) { return rank_code(row[i], i < a.keep_first || i >= nb - a.keep_last); };
  uint32_t prefix = 0;
  int need = want;                                       // still to be found among codes with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += kSelectThreads) {
      const uint32_t c = code(i);
      if (shift == 24 || (c >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(c >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // bins from the top: the one in which the need-th largest code lies
      int above = 0;
      for (int g = 7; g >= 0; --g) {
        int n = hist[g * 32 + (31 - lane)], x = n;       // lane 0 the highest bin
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, above + x >= need);
        if (hit) {
          const int first = __ffs(hit) - 1;
          if (lane == first) {
            pick[0] = g * 32 + 31 - lane;
            pick[1] = need - (above + x - n);
          }
          break;
        }
        above += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    need = pick[1];
    __syncthreads();
  }
  // codes above `prefix`, and the first `need` that equal it
  int written = 0, equal = 0;
  for (int i0 = 0; i0 < nb; i0 += kSelectThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t c = i < nb ? code(i) : 0u;
    const bool over = i < nb && c > prefix, same = i < nb && c == prefix;
    const uint32_t mo = __ballot_sync(0xffffffffu, over), ms = __ballot_sync(0xffffffffu, same);
    if (lane == 0) warp_sum[warp] = __popc(mo) << 16 | __popc(ms);
    __syncthreads();
    int before_o = 0, before_s = 0, all_o = 0, all_s = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      const int v = warp_sum[w];
      if (w < warp) { before_o += v >> 16; before_s += v & 0xFFFF; }
      all_o += v >> 16;
      all_s += v & 0xFFFF;
    }
    const uint32_t lt = (1u << lane) - 1u;
    const int o = before_o + __popc(mo & lt), sm = before_s + __popc(ms & lt);
    // `equal` of the equal codes came before this round; those past `need` are left out
    const int taken_before = min(equal + sm, need) - min(equal, need);
    if (over || (same && equal + sm < need)) out[written + o + taken_before] = i;
    written += all_o + min(equal + all_s, need) - min(equal, need);
    equal += all_s;
    __syncthreads();
  }
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t s) {
  select_kernel<<<a.T, kSelectThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
