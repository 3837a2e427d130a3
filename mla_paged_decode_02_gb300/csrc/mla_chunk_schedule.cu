// mla_chunk_schedule.cu — the on-device scheduler of the ragged chunk attention, and the merge
// of the blocks it cuts.
//
// Sequence b brings n_b = cu_q[b+1] - cu_q[b] new tokens, n_b H query rows, in blocks of 128.
// The block with rows up to token i sees v = L_b - n_b + 1 + i keys (causal; else L_b), i.e.
// ceil(v / 256) tiles: under the causal mask the blocks of one sequence differ, so each has its
// own count (an equal count for all would leave half the positions of a prompt empty). The
// blocks of all sequences are laid end to end, each as X set-up positions and its tiles, and
// worker c (a CTA pair) takes the positions [c q, (c+1) q), q = ceil(W / workers): no worker
// has more than one tile more work than another. A block that a boundary cuts becomes one unit
// per worker; the pieces leave partial outputs with their log-sum-exps, merged by the combine
// kernel below. One CTA: two block-wide scans over the sequences and over the blocks (each
// thread a contiguous range), so that the cost grows with blocks / 1024.
#include "mla_chunk.h"
#include "mla_ptx.cuh"
#include "mla_scan.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

__device__ __forceinline__ int clamp_len(int L, int max_len) { return L < 0 ? 0 : (L > max_len ? max_len : L); }

}  // namespace

__global__ void __launch_bounds__(kSchedThreads) chunk_schedule_kernel(ChunkSchedArgs a) {
  __shared__ int64_t scan_tmp[32];
  const int tid = threadIdx.x;
  griddep_wait();                          // the lengths and the workspace may be the work before's
  griddep_launch_dependents();
  // 1. blocks per sequence, and the checks of the inputs only the device can see
  const int B = a.B;
  const int chunk = (B + kSchedThreads - 1) / kSchedThreads;
  const int b0 = min(B, tid * chunk), b1 = min(B, b0 + chunk);
  int64_t mine = 0;
  uint32_t bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int s = a.cu_q[b], e = a.cu_q[b + 1], L = a.seq_lens[b];
    if (s < 0 || e < s || e > a.tokens) {
      bad |= MLA_DEVERR_CU_Q;
    } else {
      mine += ((int64_t)(e - s) * a.H + kChunkRows - 1) / kChunkRows;
    }
    if (L != clamp_len(L, a.max_len)) bad |= MLA_DEVERR_SEQ_LEN;
  }
  int64_t S;
  int64_t off = block_exclusive_scan(mine, scan_tmp, &S);
  // offsets that do not ascend within the rows of q: nothing is computed
  const bool refuse = __syncthreads_or((bad & MLA_DEVERR_CU_Q) != 0) != 0;
  const bool bad_len = __syncthreads_or((bad & MLA_DEVERR_SEQ_LEN) != 0) != 0;
  if (tid == 0) a.hdr[0] = (refuse ? MLA_DEVERR_CU_Q : 0u) | (bad_len ? MLA_DEVERR_SEQ_LEN : 0u);
  if (refuse || S == 0) {
    for (int c = tid; c <= a.workers; c += kSchedThreads) a.cta_first[c] = 0;
    if (tid == 0) a.hdr[1] = a.hdr[2] = a.hdr[3] = a.hdr[4] = 0;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    a.gbase[b] = (int32_t)off;
    off += ((int64_t)(a.cu_q[b + 1] - a.cu_q[b]) * a.H + kChunkRows - 1) / kChunkRows;
  }
  if (tid == 0) a.gbase[B] = (int32_t)S;
  __syncthreads();

  // 2. positions of the blocks, as one flattened index space
  const int64_t schunk = (S + kSchedThreads - 1) / kSchedThreads;
  const int64_t s0 = min(S, (int64_t)tid * schunk), s1 = min(S, s0 + schunk);
  int bfirst = 0;                          // the sequence of block s0: the last with gbase <= s0
  if (s0 < s1) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.gbase[mid] <= s0) lo = mid;
      else hi = mid - 1;
    }
    bfirst = lo;
  }
  // walks blocks s0 .. s1 - 1: f(s, b, first row in the sequence, rows, L, keys the first token sees, tiles)
  auto walk = [&](auto&& f) {
    int b = bfirst;
    int64_t gb = 0, ge = 0;
    int n = 0, L = 0, start = 0;
    bool have = false;
    for (int64_t s = s0; s < s1; ++s) {
      while (!have || s >= ge) {
        if (have) ++b;
        gb = a.gbase[b];
        ge = a.gbase[b + 1];
        have = true;
        start = a.cu_q[b];
        n = a.cu_q[b + 1] - start;
        L = clamp_len(a.seq_lens[b], a.max_len);
      }
      const int64_t r0 = (s - gb) * kChunkRows;
      const int64_t left = (int64_t)n * a.H - r0;
      const int rows = left < kChunkRows ? (int)left : kChunkRows;
      const int vis = a.causal ? L - n + 1 : L;
      int last = a.causal ? vis + (int)((uint32_t)(r0 + rows - 1) / (uint32_t)a.H) : L;   // rows < 2^30
      last = last < 0 ? 0 : last;
      f(b, start, r0, rows, L, vis, (last + kChunkTile - 1) / kChunkTile);
    }
  };
  int64_t sum_tiles = 0;
  walk([&](int, int, int64_t, int, int, int, int tiles) { sum_tiles += tiles > 0 ? tiles : 1; });
  int64_t W0;
  const int64_t pre_tiles = block_exclusive_scan(sum_tiles, scan_tmp, &W0);
  // X is dropped when a worker's share would be too small for it (q <= 2 X): then every
  // worker's range holds at least one tile
  int X = a.setup;
  int64_t q = (W0 + S * X + a.workers - 1) / a.workers;
  if (X > 0 && q <= 2 * (int64_t)X) {
    X = 0;
    q = (W0 + a.workers - 1) / a.workers;
  }
  // which worker a position belongs to. 64-bit divisions are several times as long: the smallest
  // call takes 17.4 us so and 18.6 us with them and a scan for each count below
  const bool small = W0 + S * X + q < (int64_t)1 << 31;
  auto worker_of = [&](int64_t p) -> int64_t { return small ? (int64_t)((uint32_t)p / (uint32_t)q) : p / q; };
  int64_t mine3 = 0;                       // units << 32 | cut blocks << 16 | partial slots
  int64_t pos = pre_tiles + s0 * X;
  walk([&](int, int, int64_t, int, int, int, int tiles) {
    const int64_t ts = pos + X;
    const int n = tiles > 0 ? tiles : 1;
    const int64_t ns = worker_of(ts + n - 1) - worker_of(ts) + 1;
    mine3 += ns << 32;
    if (ns >= 2) mine3 += (1 << 16) + ns;
    pos = ts + n;
  });
  // one scan of all three: fewer than 2^15 workers, so that their fields do not overflow
  int64_t all3;
  const int64_t before3 = block_exclusive_scan(mine3, scan_tmp, &all3);
  const int64_t n_units = all3 >> 32, n_split = (all3 >> 16) & 0xFFFF;
  int64_t unit_off = before3 >> 32, split_off = (before3 >> 16) & 0xFFFF, slot_off = before3 & 0xFFFF;
  for (int c = tid; c <= a.workers; c += kSchedThreads) a.cta_first[c] = (int32_t)n_units;
  __syncthreads();
  pos = pre_tiles + s0 * X;
  walk([&](int b, int start, int64_t r0, int rows, int L, int vis, int tiles) {
    const int64_t pre = pos, ts = pos + X;
    const int n = tiles > 0 ? tiles : 1;
    const int64_t c_lo = worker_of(ts);
    const int ns = (int)(worker_of(ts + n - 1) - c_lo + 1);
    const int32_t row0 = (int32_t)((int64_t)start * a.H + r0);
    if (ns >= 2) a.split_list[split_off++] = make_int4(row0, rows, ns, (int)slot_off);
    for (int k = 0; k < ns; ++k) {
      const int64_t c = c_lo + k;
      const int64_t p0 = ts > c * q ? ts : c * q;
      const int64_t p1 = ts + n < (c + 1) * q ? ts + n : (c + 1) * q;
      const int tb = (int)(p0 - ts), te = tiles > 0 ? (int)(p1 - ts) : 0;
      int4* u = reinterpret_cast<int4*>(a.units + unit_off);
      u[0] = make_int4(b, row0, (int32_t)r0, tb | (te << 16));
      u[1] = make_int4(ns >= 2 ? (int)slot_off + k : -1, L, vis, rows);
      // the worker's first unit: its range starts at this piece, or inside this block's set-up
      if (p0 == c * q || (k == 0 && pre <= c * q)) a.cta_first[c] = (int32_t)unit_off;
      ++unit_off;
    }
    if (ns >= 2) slot_off += ns;
    pos = ts + n;
  });
  if (tid == 0) {
    a.hdr[1] = (uint32_t)n_units;
    a.hdr[2] = (uint32_t)n_split;
    a.hdr[3] = (uint32_t)(q < 0xFFFFFFFFll ? q : 0xFFFFFFFFll);
    a.hdr[4] = (uint32_t)X;
  }
}

// Few cut rows (four warps exist for each): a warp per 128 columns of a row, lane s holding the
// weight of piece s, four pieces read at a time. The call on 16 blocks cut into 6 pieces each takes
// 64.5 us so and 66.5 us with a warp per row; with 76 cut blocks a warp per row is 1 us faster.
template <int kRows>
__device__ __forceinline__ void merge_few_rows(const ChunkCombineArgs& a, int64_t tasks, int64_t warp) {
  const int lane = threadIdx.x & 31;
  if (warp >= tasks * 4) return;
  const int4 st = a.split_list[warp / (kRows * 4)];
  const int r = (int)(warp >> 2) % kRows, col = ((int)warp & 3) * 128 + lane * 4;
  if (r >= st.y) return;
  const int ns = st.z;
  const float* plse = a.part_lse + (int64_t)st.w * kRows + r;
  const float* po = a.part_o + ((int64_t)st.w * kRows + r) * kDV + col;
  float m = -INFINITY;
  for (int s = lane; s < ns; s += 32) m = fmaxf(m, plse[(int64_t)s * kRows]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float wsum = 0.f;
  for (int s0 = 0; s0 < ns; s0 += 32) {
    const int mine = s0 + lane;
    const float ls = mine < ns ? plse[(int64_t)mine * kRows] : -INFINITY;
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
        if (ww[k] != 0.f) v[k] = *reinterpret_cast<const float4*>(po + (int64_t)(s0 + s + k) * kRows * kDV);
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
// pool among those the call read (they read page 0). A partial slot has kRows rows.
template <int kRows>
__global__ void __launch_bounds__(256) chunk_combine_kernel(ChunkCombineArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t gtid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, gstride = (int64_t)gridDim.x * blockDim.x;
  griddep_wait();
  if ((a.hdr[0] & MLA_DEVERR_CU_Q) == 0) {
    for (int64_t i = gtid; i < (int64_t)a.B * a.MB; i += gstride) {
      const int b = (int)(i / a.MB), j = (int)(i - (int64_t)b * a.MB);
      if (a.cu_q[b + 1] > a.cu_q[b] && (int64_t)j * a.P < clamp_len(a.seq_lens[b], a.max_len)) {
        const int pg = a.block_table[i];
        if (pg < 0 || pg >= a.num_pages) atomicOr(a.err, MLA_DEVERR_BLOCK_TABLE);
      }
    }
  }
  const int64_t tasks = (int64_t)a.hdr[2] * kRows;
  if (tasks * 4 <= gstride >> 5) {
    merge_few_rows<kRows>(a, tasks, gtid >> 5);
    return;
  }
  for (int64_t task = gtid >> 5; task < tasks; task += gstride >> 5) {
    const int4 st = a.split_list[task / kRows];
    const int r = (int)(task % kRows);
    if (r >= st.y) continue;
    const int ns = st.z, base = st.w;
    float m = -INFINITY;
    for (int s = 0; s < ns; ++s) m = fmaxf(m, a.part_lse[(int64_t)(base + s) * kRows + r]);
    float acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    float wsum = 0.f;
    for (int s = 0; s < ns; ++s) {
      const float ls = a.part_lse[(int64_t)(base + s) * kRows + r];
      if (ls == -INFINITY) continue;
      const float w = __expf(ls - m);
      wsum += w;
      const float4* src = reinterpret_cast<const float4*>(a.part_o + ((int64_t)(base + s) * kRows + r) * kDV) + lane * 4;
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

cudaError_t launch_chunk_combine(const ChunkCombineArgs& a, int rows, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return rows == kChunkRows ? cudaLaunchKernelEx(&cfg, chunk_combine_kernel<kChunkRows>, a)
                            : cudaLaunchKernelEx(&cfg, chunk_combine_kernel<16>, a);
}

}  // namespace mla
