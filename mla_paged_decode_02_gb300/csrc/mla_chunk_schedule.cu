// mla_chunk_schedule.cu — the on-device scheduler of the ragged chunk attention, and the merge
// of the blocks it cuts (the partition itself is in mla_chunk_schedule.cuh).
#include "mla_chunk_schedule.cuh"
#include "mla_ptx.cuh"

namespace mla {

__global__ void __launch_bounds__(kSchedThreads) chunk_schedule_kernel(ChunkSchedArgs a) {
  __shared__ int64_t scan_tmp[32];
  griddep_wait();                          // the lengths and the workspace may be the work before's
  griddep_launch_dependents();
  chunk_schedule(a, RaggedSeqs{a.seq_lens, a.cu_q, a.max_len, a.tokens}, 0u, scan_tmp);
}

// Few cut rows (four warps exist for each): a warp per 128 columns of a row, lane s holding the
// weight of piece s, four pieces read at a time. The call on 16 blocks cut into 6 pieces each takes
// 64.5 us so and 66.5 us with a warp per row; with 76 cut blocks a warp per row is 1 us faster.
__device__ __forceinline__ void merge_few_rows(const ChunkCombineArgs& a, int64_t tasks, int64_t warp) {
  const int lane = threadIdx.x & 31;
  if (warp >= tasks * 4) return;
  const int4 st = a.split_list[warp / (kChunkRows * 4)];
  const int r = (int)(warp >> 2) % kChunkRows, col = ((int)warp & 3) * 128 + lane * 4;
  if (r >= st.y) return;
  const int ns = st.z;
  const float* plse = a.part_lse + (int64_t)st.w * kChunkRows + r;
  const float* po = a.part_o + ((int64_t)st.w * kChunkRows + r) * kDV + col;
  float m = -INFINITY;
  for (int s = lane; s < ns; s += 32) m = fmaxf(m, plse[(int64_t)s * kChunkRows]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float wsum = 0.f;
  for (int s0 = 0; s0 < ns; s0 += 32) {
    const int mine = s0 + lane;
    const float ls = mine < ns ? plse[(int64_t)mine * kChunkRows] : -INFINITY;
    const float w = ls == -INFINITY ? 0.f : __expf(ls - m);
    const int n = min(32, ns - s0);
    for (int s = 0; s < n; s += 4) {
      float4 v[4];
      float ww[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ww[k] = s + k < n ? __shfl_sync(0xffffffffu, w, s + k) : 0.f;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        // a NaN weight is read: it makes the row NaN
        if (ww[k] != 0.f) v[k] = *reinterpret_cast<const float4*>(po + (int64_t)(s0 + s + k) * kChunkRows * kDV);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wsum += ww[k];
        acc.x += ww[k] * v[k].x;
        acc.y += ww[k] * v[k].y;
        acc.z += ww[k] * v[k].z;
        acc.w += ww[k] * v[k].w;
      }
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;     // a row that sees no key: zeros
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 h1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  const int64_t row = (int64_t)st.x + r;
  *reinterpret_cast<uint2*>(a.out + row * kDV + col) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  if (lane == 0 && (warp & 3) == 0) a.lse[row] = wsum == 0.f ? -INFINITY : m + logf(wsum);
}

// Merges the pieces of cut blocks, a warp per (block, row): lse = log sum_s exp(lse_s),
// out = sum_s exp(lse_s - lse) O_s; a piece in which the row sees no key has lse_s = -inf and
// weight 0. Lane l owns output columns 16 l ..; also reports block-table entries outside the
// pool among those the call read (they read page 0).
__global__ void __launch_bounds__(256) chunk_combine_kernel(ChunkCombineArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t gtid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, gstride = (int64_t)gridDim.x * blockDim.x;
  griddep_wait();
  if ((a.hdr[0] & MLA_DEVERR_CU_Q) == 0) {
    for (int64_t i = gtid; i < (int64_t)a.B * a.MB; i += gstride) {
      const int b = (int)(i / a.MB), j = (int)(i - (int64_t)b * a.MB);
      if (a.cu_q[b + 1] > a.cu_q[b] && (int64_t)j * a.P < RaggedSeqs::clamp_len(a.seq_lens[b], a.max_len)) {
        const int pg = a.block_table[i];
        if (pg < 0 || pg >= a.num_pages) atomicOr(a.err, MLA_DEVERR_BLOCK_TABLE);
      }
    }
  }
  const int64_t tasks = (int64_t)a.hdr[2] * kChunkRows;
  if (tasks * 4 <= gstride >> 5) {
    merge_few_rows(a, tasks, gtid >> 5);
    return;
  }
  for (int64_t task = gtid >> 5; task < tasks; task += gstride >> 5) {
    const int4 st = a.split_list[task / kChunkRows];
    const int r = (int)(task % kChunkRows);
    if (r >= st.y) continue;
    const int ns = st.z, base = st.w;
    float m = -INFINITY;
    for (int s = 0; s < ns; ++s) m = fmaxf(m, a.part_lse[(int64_t)(base + s) * kChunkRows + r]);
    float acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    float wsum = 0.f;
    for (int s = 0; s < ns; ++s) {
      const float ls = a.part_lse[(int64_t)(base + s) * kChunkRows + r];
      if (ls == -INFINITY) continue;
      const float w = __expf(ls - m);
      wsum += w;
      const float4* src = reinterpret_cast<const float4*>(a.part_o + ((int64_t)(base + s) * kChunkRows + r) * kDV) + lane * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = src[k];
        acc[4 * k + 0] += w * v.x;
        acc[4 * k + 1] += w * v.y;
        acc[4 * k + 2] += w * v.z;
        acc[4 * k + 3] += w * v.w;
      }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;   // a row that sees no key: zeros
    uint32_t packed[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      packed[k] = *reinterpret_cast<uint32_t*>(&h);
    }
    const int64_t row = (int64_t)st.x + r;
    uint4* dst = reinterpret_cast<uint4*>(a.out + row * kDV) + lane * 2;
    dst[0] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    dst[1] = make_uint4(packed[4], packed[5], packed[6], packed[7]);
    if (lane == 0) a.lse[row] = wsum == 0.f ? -INFINITY : m + logf(wsum);
  }
}

cudaError_t launch_chunk_schedule(const ChunkSchedArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kSchedThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_schedule_kernel, a);
}

cudaError_t launch_chunk_combine(const ChunkCombineArgs& a, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_combine_kernel, a);
}

}  // namespace mla
