// mla_sparse_plan.cu — the plan of a sparse attention.
//
// A token attends over the keys it sees in a set of blocks of its sequence. To the chunk attention's
// kernels that is a sequence of its own, with one new token, pages of `block` rows and a page table
// that names the chosen blocks in ascending order: only its last page can hold keys that the token
// does not see, so a length says which keys count. The plan makes that table and those lengths,
// whatever the order of the caller's list: the chosen blocks are marked in a bit set, so that an index
// given twice counts once, and those without a key that the token sees (negative ones among them) are
// left out.
//
// One cluster of eight CTAs: a warp takes a token at a time, then the first CTA partitions the tokens'
// keys over the attention's workers, as the chunk attention's scheduler does.
#include "mla_chunk_schedule.cuh"
#include "mla_index.h"
#include "mla_ptx.cuh"
#include "mla_ragged.cuh"

namespace mla {
namespace {

// Token t as a sequence of its own; rows [first, last) belong to sequences.
struct TokenSeqs {
  static constexpr bool kMayFlagTable = true;
  const int32_t* lens;
  int first, last;
  __device__ __forceinline__ int start(int t) const { return t; }
  __device__ __forceinline__ int count(int t) const { return t >= first && t < last ? 1 : 0; }
  __device__ __forceinline__ int len(int t) const { return lens[t]; }
  __device__ __forceinline__ uint32_t errors(int) const { return 0u; }
};

}  // namespace

__global__ void __launch_bounds__(kSchedThreads, 1) sparse_plan_kernel(SparsePlanArgs a, int warps) {
  extern __shared__ uint32_t sets[];                     // [warps][words]
  __shared__ int64_t scan_tmp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank();
  griddep_wait();                          // the inputs and the workspace may be the work before's
  griddep_launch_dependents();
  uint32_t bad = 0;
  for (int b = rank * kSchedThreads + threadIdx.x; b < a.B; b += kPlanCtas * kSchedThreads)
    bad |= ragged_errors(a.cu_q, a.seq_lens, b, a.T, a.max_len);
  if (warp < warps) {
    uint32_t* set = sets + (size_t)warp * a.words;
    const int per_page = a.P / a.block;
    for (int t = rank * warps + warp; t < a.T; t += kPlanCtas * warps) {
      const int b = sequence_of(a.cu_q, a.B, t, lane);
      int seen = 0;
      if (b >= 0) {
        const int L = max(0, min(a.seq_lens[b], a.max_len));
        seen = keys_seen(t, a.cu_q[b], a.cu_q[b + 1], L, a.causal);
      }
      const int nb = (seen + a.block - 1) / a.block, nw = (nb + 31) >> 5;
      for (int w = lane; w < nw; w += 32) set[w] = 0u;
      __syncwarp();
      const int32_t* chosen = a.selected + (int64_t)t * a.K;
      for (int k = lane; k < a.K && nb > 0; k += 32) {
        const int c = chosen[k];
        if (c >= 0 && c < nb) atomicOr(set + (c >> 5), 1u << (c & 31));
      }
      __syncwarp();
      int32_t* row = a.table + (int64_t)t * a.width;
      const int32_t* pages = a.block_table + (int64_t)(b < 0 ? 0 : b) * a.MB;
      int total = 0;
      for (int w0 = 0; w0 < nw; w0 += 32) {
        uint32_t word = w0 + lane < nw ? set[w0 + lane] : 0u;
        const int n = __popc(word);
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += y;
        }
        const int all = __shfl_sync(0xffffffffu, at, 31);
        at += total - n;
        total += all;
        while (word) {
          const int c = (w0 + lane) * 32 + __ffs(word) - 1;
          word &= word - 1;
          int pg = pages[c / per_page];
          if (pg < 0 || pg >= a.num_pages) {             // reads page 0, as elsewhere
            bad |= MLA_DEVERR_BLOCK_TABLE;
            pg = 0;
          }
          row[at++] = pg * per_page + c % per_page;
        }
      }
      if (lane == 0) {
        const bool partial = nb > 0 && (set[(nb - 1) >> 5] >> ((nb - 1) & 31) & 1u) != 0u;
        a.lens[t] = total * a.block - (partial ? nb * a.block - seen : 0);
      }
      __syncwarp();
    }
  }
  bad = (__syncthreads_or((bad & MLA_DEVERR_CU_Q) != 0) ? MLA_DEVERR_CU_Q : 0u) |
        (__syncthreads_or((bad & MLA_DEVERR_SEQ_LEN) != 0) ? MLA_DEVERR_SEQ_LEN : 0u) |
        (__syncthreads_or((bad & MLA_DEVERR_BLOCK_TABLE) != 0) ? MLA_DEVERR_BLOCK_TABLE : 0u);
  if (threadIdx.x == 0) a.flags[rank] = bad;
  cluster_sync();                          // tables, lengths and flags of all CTAs
  if (rank != 0) return;
  bad = threadIdx.x < kPlanCtas ? a.flags[threadIdx.x] : 0u;
  chunk_schedule(a.sched, TokenSeqs{a.lens, a.cu_q[0], a.cu_q[a.B]}, bad, scan_tmp);
}

cudaError_t launch_sparse_plan(const SparsePlanArgs& a, cudaStream_t s) {
  // as many warps as have room for their sets: 32 up to 48 K blocks
  constexpr int kRoom = 200 * 1024;
  int warps = kRoom / (a.words * 4);
  warps = warps > 32 ? 32 : warps;
  const size_t smem = (size_t)warps * a.words * 4;
  cudaError_t e = cudaFuncSetAttribute(sparse_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kSchedThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPlanCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sparse_plan_kernel, a, warps);
}

}  // namespace mla
