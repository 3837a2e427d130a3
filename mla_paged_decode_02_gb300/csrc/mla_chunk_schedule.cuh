// mla_chunk_schedule.cuh — the partition of a ragged batch's blocks over the chunk attention's
// workers, by one CTA of 1024 threads (the scheduler of the chunk attention and the plan of the
// sparse attention, which differ in where a sequence's rows and keys come from).
//
// Sequence b brings n_b = cu_q[b+1] - cu_q[b] new tokens, n_b H query rows, in blocks of 128.
// The block with rows up to token i sees v = L_b - n_b + 1 + i keys (causal; else L_b), i.e.
// ceil(v / 256) tiles: under the causal mask the blocks of one sequence differ, so each has its
// own count (an equal count for all would leave half the positions of a prompt empty). The
// blocks of all sequences are laid end to end, each as X set-up positions and its tiles, and
// worker c (a CTA pair) takes the positions [c q, (c+1) q), q = ceil(W / workers): no worker
// has more than one tile more work than another. A block that a boundary cuts becomes one unit
// per worker; the pieces leave partial outputs with their log-sum-exps, merged by the combine
// kernel. One CTA: two block-wide scans over the sequences and over the blocks (each
// thread a contiguous range), so that the cost grows with blocks / 1024.
#pragma once
#include "mla_chunk.h"
#include "mla_scan.cuh"
#include "../../include/mla.h"

namespace mla {

// The sequences as the caller gives them: rows cu_q[b] .. cu_q[b + 1], clamped lengths.
struct RaggedSeqs {
  static constexpr bool kMayFlagTable = false;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int max_len, tokens;
  __device__ __forceinline__ static int clamp_len(int L, int max_len) { return L < 0 ? 0 : (L > max_len ? max_len : L); }
  __device__ __forceinline__ int start(int b) const { return cu_q[b]; }
  __device__ __forceinline__ int count(int b) const { return cu_q[b + 1] - cu_q[b]; }
  __device__ __forceinline__ int len(int b) const { return clamp_len(seq_lens[b], max_len); }
  __device__ __forceinline__ uint32_t errors(int b) const {
    const int s = cu_q[b], e = cu_q[b + 1], L = seq_lens[b];
    return (s < 0 || e < s || e > tokens ? MLA_DEVERR_CU_Q : 0u) | (L != clamp_len(L, max_len) ? MLA_DEVERR_SEQ_LEN : 0u);
  }
};

// `bad`: error bits that this thread has found already.
template <class Seqs>
__device__ __forceinline__ void chunk_schedule(const ChunkSchedArgs& a, const Seqs& seqs, uint32_t bad, int64_t* scan_tmp) {
  const int tid = threadIdx.x;
  // 1. blocks per sequence, and the checks of the inputs only the device can see
  const int B = a.B;
  const int chunk = (B + kSchedThreads - 1) / kSchedThreads;
  const int b0 = min(B, tid * chunk), b1 = min(B, b0 + chunk);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const uint32_t e = seqs.errors(b);
    bad |= e;
    if ((e & MLA_DEVERR_CU_Q) == 0) mine += ((int64_t)seqs.count(b) * a.H + kChunkRows - 1) / kChunkRows;
  }
  int64_t S;
  int64_t off = block_exclusive_scan(mine, scan_tmp, &S);
  // offsets that do not ascend within the rows of q: nothing is computed
  const bool refuse = __syncthreads_or((bad & MLA_DEVERR_CU_Q) != 0) != 0;
  const bool bad_len = __syncthreads_or((bad & MLA_DEVERR_SEQ_LEN) != 0) != 0;
  const bool bad_table = Seqs::kMayFlagTable && __syncthreads_or((bad & MLA_DEVERR_BLOCK_TABLE) != 0) != 0;
  if (tid == 0)
    a.hdr[0] = (refuse ? MLA_DEVERR_CU_Q : 0u) | (bad_len ? MLA_DEVERR_SEQ_LEN : 0u) | (bad_table ? MLA_DEVERR_BLOCK_TABLE : 0u);
  if (refuse || S == 0) {
    for (int c = tid; c <= a.workers; c += kSchedThreads) a.cta_first[c] = 0;
    if (tid == 0) a.hdr[1] = a.hdr[2] = a.hdr[3] = a.hdr[4] = 0;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    a.gbase[b] = (int32_t)off;
    off += ((int64_t)seqs.count(b) * a.H + kChunkRows - 1) / kChunkRows;
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
        start = seqs.start(b);
        n = seqs.count(b);
        L = seqs.len(b);
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

}  // namespace mla
