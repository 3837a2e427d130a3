// mla_index_scores.cu — scores of the blocks of a ragged batch's contexts.
//
// For token t, key j it sees and block c of `block` keys:
//   s_j = scale_j sum_h w_h max(0, q_h . k_j),   S_c = max over the seen keys j of block c of s_j,
// -inf for a block without one; a NaN counts as -inf.
#include <cuda_fp8.h>
#include "mla_index.h"
#include "mla_ragged.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

// an order-preserving code of a float, so that maxima can be taken as integers
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
// max(0, x) that keeps a NaN
__device__ __forceinline__ float positive(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

}  // namespace

// A CTA takes one token and `per` blocks; a thread a key.
__global__ void __launch_bounds__(128) index_scores_kernel(IndexScoreArgs a, int per) {
  extern __shared__ float sq[];                          // [H][128] and the weights
  __shared__ int best[16];
  const int lane = threadIdx.x & 31, t = blockIdx.x;
  const int limit = min(a.max_len, a.MB * a.P);
  for (int b = t * 128 + threadIdx.x; blockIdx.y == 0 && b < a.B; b += gridDim.x * 128) {
    const uint32_t bad = ragged_errors(a.cu_q, a.seq_lens, b, a.T, a.max_len);
    if (bad && a.err) atomicOr(a.err, bad);
  }
  const int b = sequence_of(a.cu_q, a.B, t, lane);
  if (b < 0) return;
  const int L = max(0, min(a.seq_lens[b], limit));
  const int seen = keys_seen(t, a.cu_q[b], a.cu_q[b + 1], L, a.causal);
  float* sw = sq + a.H * kDIndex;
  for (int i = threadIdx.x; i < a.H * kDIndex; i += 128) {
    __nv_fp8_e4m3 e;
    e.__x = a.q[(int64_t)t * a.H * kDIndex + i];
    sq[i] = float(e);
  }
  for (int i = threadIdx.x; i < a.H; i += 128) sw[i] = a.w[(int64_t)t * a.H + i];
  if (threadIdx.x < 16) best[threadIdx.x] = ordered(-INFINITY);
  __syncthreads();
  const int c0 = blockIdx.y * per;
  const int64_t k0 = (int64_t)c0 * a.block;
  const int64_t k1 = min((int64_t)seen, k0 + (int64_t)per * a.block);
  for (int64_t j = k0 + threadIdx.x; j < k1; j += 128) {
    int pg = a.block_table[(int64_t)b * a.MB + j / a.P];
    if (pg < 0 || pg >= a.num_pages) {
      pg = 0;
      if (a.err) atomicOr(a.err, MLA_DEVERR_BLOCK_TABLE);
    }
    const int64_t row = (int64_t)pg * a.P + j % a.P;
    float sum = 0.f;
    for (int h = 0; h < a.H; ++h) {
      float d = 0.f;
      for (int i = 0; i < kDIndex; ++i) {
        __nv_fp8_e4m3 e;
        e.__x = a.cache[row * kDIndex + i];
        d += float(e) * sq[h * kDIndex + i];
      }
      sum += sw[h] * positive(d);
    }
    sum *= a.scale[row];
    if (sum > -INFINITY) atomicMax(&best[(j - k0) / a.block], ordered(sum));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < per && c0 + i < a.C; i += 128) a.out[(int64_t)t * a.C + c0 + i] = from_ordered(best[i]);
}

cudaError_t launch_index_scores(const IndexScoreArgs& a, cudaStream_t s) {
  const int per = a.block < 128 ? 128 / a.block : 1;
  const int smem = (a.H * kDIndex + a.H) * 4;
  cudaError_t e = cudaFuncSetAttribute(index_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  index_scores_kernel<<<dim3(a.T, (a.C + per - 1) / per), 128, smem, s>>>(a, per);
  return cudaGetLastError();
}

}  // namespace mla
