// mla_sparse_plan.cu — the plan of a sparse attention.
//
// A token attends over the keys it sees in a set of blocks of its sequence. To the chunk attention's
// kernels that is a sequence of its own, with one new token, pages of `block` rows and a page table
// that names the chosen blocks in ascending order: only its last page can hold keys that the token
// does not see, so a length says which keys count. The plan makes that table and those lengths,
// whatever the order of the caller's list: blocks without a key that the token sees (negative ones among
// them) are left out, and a list that does not ascend goes through a bit set, so that an index
// given twice counts once.
//
// Then the tokens' keys are shared out. A token's H rows are ceil(H / 128) blocks of up to 128 rows with equally
// many tiles of 256 keys (for the decode kernel one block, and tiles of 128); laid end to end, X set-up positions
// and the tiles for each, worker c (a CTA pair; an SM) takes positions [c q, (c + 1) q), q = ceil(all / workers).
// A block that a boundary cuts becomes one unit per worker. (The partition of the chunk scheduler, without its
// search for the sequence of a block: here a block's number says which token it belongs to.) Where a share holds
// six blocks or more, blocks stay whole and go to the worker in whose share their middle lies: a worker then has
// up to half a block more, and nothing is merged. us, whole / cut, 2041 keys a token: E4M3, 16 heads, 1024 tokens
// 239 / 286, 2048 468 / 552; 128 heads, 512 tokens, bf16 185 / 194, E4M3 192 / 193; 1024, bf16, 366 / 367, with 512 keys
// 134 / 138. Shares of five blocks, 384 tokens x 128 heads: bf16 157 / 152, E4M3 160 / 154; of three, 512 x 16, E4M3,
// 140 / 151.
// With no more blocks than workers, each worker has a piece of one
// block where such pieces need not be much longer than q: starting on a second block costs a worker about two
// tiles (16 heads, E4M3, 2041 keys: 48 tokens 28.8 us against 33.8, 64 33.1 against 35.4, 152 55 against 61; 128
// heads, bf16, 64 tokens 54 against 65; those with uneven lengths from 4 less to 1 more).
//
// One cluster of eight CTAs: a warp takes a token at a time and sends its length to the first CTA's shared
// memory, where the partition is made. Bound by latency: the list, lengths and offsets are read at once,
// then the page numbers; after a cluster barrier two scans by as many warps as there are 32 tokens. What ran
// all 32 warps through 64-bit arithmetic took 6.5 us for 2 to 64 tokens and 10 for 512, more than half of it
// in the partition; calls are 1 us (tiny ones) to 11 us (512 tokens) faster now. A single CTA for few tokens
// is no faster.
#include <type_traits>
#include "mla_index.h"
#include "mla_ptx.cuh"
#include "mla_ragged.cuh"

namespace mla {
namespace {

constexpr int kSchedThreads = 1024;
constexpr int kRoom = 220 * 1024;          // shared memory for lengths and sets
constexpr int kPieces = 8;                 // sizes of pieces that are tried (a power of two)
constexpr int kPlanLens = 8192;            // tokens whose lengths fit the first CTA's shared memory

// tiles of 256 keys (a block that sees no key has one, in which its zeros are written), or of 128 for the
// decode kernel, which has no part in a token without keys
template <bool kFew>
__device__ __forceinline__ int tiles_of(int len) {
  if (kFew) return (len + kTileTokens - 1) / kTileTokens;
  return len > 0 ? (len + kChunkTile - 1) / kChunkTile : 1;
}

// Exclusive prefix sum over the first `warps` warps, which alone take part.
__device__ __forceinline__ int64_t warps_exclusive_scan(int64_t v, int64_t* tmp, int64_t* total, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  int64_t before = 0, all = __shfl_sync(0xffffffffu, x, 31);
  if (warps > 1) {
    if (lane == 31) tmp[warp] = x;
    named_bar_sync(1, 32 * warps);
    int64_t w = lane < warps ? tmp[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    before = warp > 0 ? before : 0;
    named_bar_sync(1, 32 * warps);           // tmp may be written again
  }
  *total = all;
  return before + x - v;
}

}  // namespace

// kFew: for the decode kernel (up to 16 rows), else for the chunk attention's. kSmall: positions fit 32 bits,
// which makes the code that runs once per launch, from instruction cache misses, a good deal shorter.
template <bool kFew, bool kSmall>
__global__ void __launch_bounds__(kSchedThreads, 1) sparse_plan_kernel(SparsePlanArgs a, int warps) {
  extern __shared__ int32_t plan_smem[];   // [T <= kPlanLens] lengths, then [warps][words] sets
  __shared__ int64_t scan_tmp[32];
  __shared__ uint32_t flags_s[kPlanCtas], bad_s;
  __shared__ int pieces_s[kPieces];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const uint32_t rank = cluster_ctarank();
  const bool near = a.T <= kPlanLens;
  // (the first CTA has to run before its shared memory is written)
  if (tid == 0) bad_s = 0u;
  if (tid < kPieces) pieces_s[tid] = 0;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  griddep_wait();                          // the inputs and the workspace may be the work before's
  griddep_launch_dependents();
  uint32_t bad = 0;
  for (int b = rank * kSchedThreads + tid; b < a.B; b += kPlanCtas * kSchedThreads)
    bad |= ragged_errors(a.cu_q, a.seq_lens, b, a.T, a.max_len);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  bool none = false;                       // a token of this warp's has no key
  const uint32_t lens_of_first = map_to_rank(smem_u32(plan_smem), 0);
  if (warp < warps) {
    uint32_t* set = reinterpret_cast<uint32_t*>(plan_smem) + (near ? a.T : 0) + (size_t)warp * a.words;
    const int per_page = a.P / a.block;
    for (int t = rank + kPlanCtas * warp; t < a.T; t += kPlanCtas * warps) {
      // at once: the list, and what is needed if sequence t is the token's
      const int32_t* chosen = a.selected + (int64_t)t * a.K;
      const int first32 = lane < a.K ? chosen[lane] : -1;
      const bool guess = t < a.B;
      int start = guess ? a.cu_q[t] : 0, end = guess ? a.cu_q[t + 1] : 0, L = guess ? a.seq_lens[t] : 0;
      int b = t;
      if (!(guess && start == t && end == t + 1)) {
        b = sequence_of(a.cu_q, a.B, t, lane);
        if (b >= 0) {
          start = a.cu_q[b];
          end = a.cu_q[b + 1];
          L = a.seq_lens[b];
        }
      }
      const int seen = b < 0 ? 0 : keys_seen(t, start, end, max(0, min(L, a.max_len)), a.causal);
      const int nb = (seen + a.block - 1) / a.block;
      int32_t* row = a.table + (int64_t)t * a.width;
      const int32_t* pages = a.block_table + (int64_t)(b < 0 ? 0 : b) * a.MB;
      auto put = [&](int at, int c) {
        const int page = per_page == 1 ? c : c / per_page;
        int pg = pages[page];
        if (pg < 0 || pg >= a.num_pages) {               // reads page 0, as elsewhere
          bad |= MLA_DEVERR_BLOCK_TABLE;
          pg = 0;
        }
        row[at] = pg * per_page + (c - page * per_page);
      };
      int total = 0, top = -1;                           // blocks so far, the largest of them
      bool ascends = true;
      for (int k0 = 0; k0 < a.K && nb > 0; k0 += 32) {
        const int c = k0 == 0 ? first32 : k0 + lane < a.K ? chosen[k0 + lane] : -1;
        const bool valid = c >= 0 && c < nb;
        const uint32_t all = __ballot_sync(0xffffffffu, valid), lower = all & ((1u << lane) - 1u);
        const int other = __shfl_sync(0xffffffffu, c, lower != 0 ? 31 - __clz(lower) : 0);
        ascends = __all_sync(0xffffffffu, !valid || c > (lower != 0 ? other : top));
        if (!ascends) break;
        if (valid) put(total + __popc(lower), c);
        if (all != 0) top = __shfl_sync(0xffffffffu, c, 31 - __clz(all));
        total += __popc(all);
      }
      if (!ascends) {
        const int nw = (nb + 31) >> 5;
        for (int w = lane; w < nw; w += 32) set[w] = 0u;
        __syncwarp();
        for (int k = lane; k < a.K; k += 32) {
          const int c = chosen[k];
          if (c >= 0 && c < nb) atomicOr(set + (c >> 5), 1u << (c & 31));
        }
        __syncwarp();
        total = 0;
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
          for (; word != 0; word &= word - 1) put(at++, (w0 + lane) * 32 + __ffs(word) - 1);
        }
        top = (set[(nb - 1) >> 5] >> ((nb - 1) & 31) & 1u) != 0u ? nb - 1 : -1;
        __syncwarp();
      }
      if (lane == 0) {
        const int len = total * a.block - (nb > 0 && top == nb - 1 ? nb * a.block - seen : 0);
        if (near) st_cluster_u32(lens_of_first + 4 * t, (uint32_t)len);
        else a.lens[t] = len;
        if (kFew) a.batch_info[t] = make_int4(0, 0, len, 0);
      }
      none |= total == 0;
    }
  }
  if (bad != 0) atomicOr(&bad_s, bad);
  __syncthreads();
  bad = bad_s;
  if (tid < kPlanCtas) st_cluster_u32(map_to_rank(smem_u32(flags_s + rank), tid), bad);
  const int first = a.cu_q[0], last = a.cu_q[a.B];
  cluster_sync();                          // tables, lengths and flags of all CTAs
  const ChunkSchedArgs& s = a.sched;
  bad = 0;
#pragma unroll
  for (int i = 0; i < kPlanCtas; ++i) bad |= flags_s[i];
  if (kFew && none && (bad & MLA_DEVERR_CU_Q) == 0) {
    // tokens without keys get their results here
    for (int t = rank + kPlanCtas * warp; t < a.T; t += kPlanCtas * warps) {
      if (t < first || t >= last || a.batch_info[t].z != 0) continue;
      uint4* out = reinterpret_cast<uint4*>(a.out + (int64_t)t * s.H * kDV);
      for (int i = lane; i < s.H * (kDV / 8); i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int i = lane; i < s.H; i += 32) a.lse[(int64_t)t * s.H + i] = -INFINITY;
    }
  }
  if (rank != 0) return;
  if (tid == 0) s.hdr[0] = bad;
  // offsets that do not ascend within the rows of q: nothing is computed
  if ((bad & MLA_DEVERR_CU_Q) != 0 || last <= first) {
    for (int c = tid; c <= s.workers; c += kSchedThreads) s.cta_first[c] = 0;
    if (tid == 0) s.hdr[1] = s.hdr[2] = s.hdr[3] = s.hdr[4] = 0;
    return;
  }
  // a token to a thread, as long as there are threads; the other warps are done
  const int tokens = last - first, scanning = min(kSchedThreads / 32, (tokens + 31) / 32), threads = 32 * scanning;
  if (warp >= scanning) return;
  const int G = kFew ? 1 : (s.H + kChunkRows - 1) / kChunkRows;   // blocks of a token
  auto len_of = [&](int t) { return near ? plan_smem[t] : a.lens[t]; };
  // a thread takes neighbouring tokens
  const int chunk = (tokens + threads - 1) / threads;
  const int t0 = first + min(tokens, tid * chunk), t1 = min(last, t0 + chunk);
  int64_t mine = 0;                        // tokens with tiles << 40 | tiles
  for (int t = t0; t < t1; ++t) {
    const int n = tiles_of<kFew>(len_of(t));
    mine += n > 0 ? ((int64_t)1 << 40) + n : 0;
  }
  int64_t all;
  const int64_t before = warps_exclusive_scan(mine, scan_tmp, &all, scanning), kTiles = ((int64_t)1 << 40) - 1;
  using Pos = std::conditional_t<kSmall, uint32_t, int64_t>;
  const Pos W = (Pos)(all & kTiles) * G, S = (Pos)(all >> 40) * G, workers = (Pos)s.workers;
  // X is dropped when a worker's share would be too small for it (q <= 2 X): then every worker's range
  // holds at least one tile
  Pos X = (Pos)s.setup, q = (W + S * X + workers - 1) / workers;
  if (X > 0 && q <= 2 * X) {
    X = 0;
    q = (W + workers - 1) / workers;
  }
  if (q == 0) q = 1;                       // (no keys at all)
  const Pos first_block = (Pos)(before >> 40) * G, pos0 = (Pos)(before & kTiles) * G + first_block * X;
  // a unit: tiles [tb, te) of block g of token t, for the attention kernels
  auto put_unit = [&](Pos unit, int t, int g, int len, int tb, int te, int slot) {
    if (kFew) {
      reinterpret_cast<int4*>(s.units)[unit] = make_int4(t, 0, tb | (te << 16), slot);
    } else {
      const int r0 = g * kChunkRows;
      int4* u = reinterpret_cast<int4*>(s.units + unit);
      u[0] = make_int4(t, t * s.H + r0, r0, len > 0 ? tb | (te << 16) : 0);
      u[1] = make_int4(slot, len, len, min(kChunkRows, s.H - r0));
    }
  };
  auto put_header = [&](Pos units, uint32_t cut) {
    if (tid != 0) return;
    s.hdr[1] = (uint32_t)units;
    s.hdr[2] = cut;
    s.hdr[3] = (uint32_t)q;
    s.hdr[4] = (uint32_t)X;
  };
  if (q >= 6 * ((Pos)tiles_of<kFew>(a.width * a.block) + X)) {
    for (int c = tid; c <= s.workers; c += threads) s.cta_first[c] = (int32_t)S;
    put_header(S, 0u);
    named_bar_sync(1, threads);
    Pos pos = pos0, unit = first_block, last_worker = ~(Pos)0;
    // the worker of the block before (of the last token before that has tiles)
    for (int t = t0 - 1; t >= first && t0 < t1; --t) {
      const Pos n = tiles_of<kFew>(len_of(t));
      if (n == 0) continue;
      last_worker = (pos0 - (X + n) + (X + n) / 2) / q;
      break;
    }
    for (int t = t0; t < t1; ++t) {
      const int len = len_of(t);
      const Pos n = tiles_of<kFew>(len);
      for (int g = 0; g < G && n > 0; ++g, ++unit) {
        const Pos c = (pos + (X + n) / 2) / q;
        put_unit(unit, t, g, len, 0, (int)n, -1);
        if (c != last_worker) s.cta_first[c] = (int32_t)unit;
        last_worker = c;
        pos += X + n;
      }
    }
    return;
  }
  if (S <= workers && q > 1 && chunk == 1) {
    // Pieces of one block each, of up to p tiles: the smallest p of a few for which there are no more pieces
    // than workers, if it is not much above q. (lo > 1, as X was dropped or q > 2 X. Quotients by an inverse
    // that one lane computes for each p, exact for tiles x p < 2^32.)
    const int lo = (int)((W + workers - 1) / workers), step = 1 + lo / 16;
    const uint32_t inverse = 0xFFFFFFFFu / (uint32_t)(lo + (lane & (kPieces - 1)) * step) + 1u;
    const int len = t0 < t1 ? len_of(t0) : 0, n = t0 < t1 ? tiles_of<kFew>(len) : 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t ns = __umulhi((uint32_t)(n + lo + i * step - 1), __shfl_sync(0xffffffffu, inverse, i));
      const int sum = __reduce_add_sync(0xffffffffu, (int)ns);
      if (lane == 0) atomicAdd(pieces_s + i, sum);
    }
    named_bar_sync(1, threads);
    const int count = pieces_s[lane & (kPieces - 1)] * G;
    const int best = __ffs(__ballot_sync(0xffffffffu, count <= s.workers)) - 1, p = lo + best * step;
    if (best >= 0 && p <= (int)q + s.setup / 2) {
      const int ns = (int)__umulhi((uint32_t)(n + p - 1), __shfl_sync(0xffffffffu, inverse, best));
      // units << 32 | cut blocks << 16 | partial slots
      int64_t all3;
      const int64_t mine3 = G * (((int64_t)ns << 32) + (ns >= 2 ? (1 << 16) + (int64_t)ns : 0));
      const int64_t before3 = warps_exclusive_scan(mine3, scan_tmp, &all3, scanning);
      const int n_units = (int)(all3 >> 32);
      int unit = (int)(before3 >> 32), split = (int)(before3 >> 16) & 0xFFFF, slot = (int)before3 & 0xFFFF;
      for (int c = tid; c <= s.workers; c += threads) s.cta_first[c] = min(c, n_units);
      put_header((Pos)n_units, (uint32_t)(all3 >> 16) & 0xFFFFu);
      for (int g = 0; g < G && n > 0; ++g) {
        const int r0 = g * kChunkRows;
        if (ns >= 2) s.split_list[split++] = make_int4(t0 * s.H + r0, min(kChunkRows, s.H - r0), ns, slot);
#pragma unroll 1
        for (int tb = 0; tb < n; tb += p, ++unit) put_unit((Pos)unit, t0, g, len, tb, min(n, tb + p), ns >= 2 ? slot++ : -1);
      }
      return;
    }
  }
  Pos pos = pos0;
  int64_t mine3 = 0;                       // units << 32 | cut blocks << 16 | partial slots (as the chunk scheduler)
  for (int t = t0; t < t1; ++t) {
    const Pos n = tiles_of<kFew>(len_of(t));
    for (int g = 0; g < G && n > 0; ++g) {
      const Pos ts = pos + X, ns = (ts + n - 1) / q - ts / q + 1;
      mine3 += ((int64_t)ns << 32) + (ns >= 2 ? (1 << 16) + (int64_t)ns : 0);
      pos = ts + n;
    }
  }
  int64_t all3;
  const int64_t before3 = warps_exclusive_scan(mine3, scan_tmp, &all3, scanning);
  const Pos n_units = (Pos)(all3 >> 32);
  Pos unit = (Pos)(before3 >> 32);
  int split = (int)(before3 >> 16) & 0xFFFF, slot = (int)before3 & 0xFFFF;
  for (int c = tid; c <= s.workers; c += threads) s.cta_first[c] = (int32_t)n_units;
  put_header(n_units, (uint32_t)(all3 >> 16) & 0xFFFFu);
  named_bar_sync(1, threads);
  pos = pos0;
  for (int t = t0; t < t1; ++t) {
    const int len = len_of(t);
    const Pos n = tiles_of<kFew>(len);
    for (int g = 0; g < G && n > 0; ++g) {
      const Pos pre = pos, ts = pos + X, c0 = ts / q;
      const int ns = (int)((ts + n - 1) / q - c0 + 1);
      if (ns >= 2) {
        const int r0 = g * kChunkRows;
        s.split_list[split++] = make_int4(t * s.H + r0, min(kChunkRows, s.H - r0), ns, slot);
      }
      Pos edge = c0 * q;                   // where the worker's range starts
      for (int k = 0; k < ns; ++k, ++unit, edge += q) {
        const Pos p0 = ts > edge ? ts : edge, p1 = ts + n < edge + q ? ts + n : edge + q;
        put_unit(unit, t, g, len, (int)(p0 - ts), (int)(p1 - ts), ns >= 2 ? slot + k : -1);
        // the worker's first unit: its range starts at this piece, or inside this block's set-up
        if (p0 == edge || (k == 0 && pre <= edge)) s.cta_first[c0 + k] = (int32_t)unit;
      }
      if (ns >= 2) slot += ns;
      pos = ts + n;
    }
  }
}

cudaError_t sparse_plan_prepare() {
  for (auto* kernel : {sparse_plan_kernel<false, false>, sparse_plan_kernel<false, true>, sparse_plan_kernel<true, false>,
                       sparse_plan_kernel<true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_sparse_plan(const SparsePlanArgs& a, cudaStream_t s) {
  // as many warps as have room for their sets: 32 for contexts up to 48 K blocks
  const int lens = a.T <= kPlanLens ? a.T : 0;
  int warps = (kRoom - lens * 4) / (a.words * 4);
  warps = warps > 32 ? 32 : warps;
  const size_t smem = (size_t)lens * 4 + (size_t)warps * a.words * 4;
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
  // the most positions there can be, and a share more
  const int64_t tile = a.few ? kTileTokens : kChunkTile, G = a.few ? 1 : (a.sched.H + kChunkRows - 1) / kChunkRows;
  const int64_t most = (int64_t)a.T * G * (((int64_t)a.width * a.block + tile - 1) / tile + 1 + a.sched.setup);
  const bool small = 2 * most + a.sched.workers < (int64_t)1 << 31;
  return a.few ? (small ? cudaLaunchKernelEx(&cfg, sparse_plan_kernel<true, true>, a, warps)
                        : cudaLaunchKernelEx(&cfg, sparse_plan_kernel<true, false>, a, warps))
               : (small ? cudaLaunchKernelEx(&cfg, sparse_plan_kernel<false, true>, a, warps)
                        : cudaLaunchKernelEx(&cfg, sparse_plan_kernel<false, false>, a, warps));
}

}  // namespace mla
