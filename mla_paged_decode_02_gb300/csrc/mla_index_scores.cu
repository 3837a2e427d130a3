// mla_index_scores.cu — scores of the blocks of a ragged batch's contexts (sm_103a, tcgen05).
//
// For token t, key j it sees and block c of `block` keys:
//   s_j = scale_j sum_h w_h max(0, q_h . k_j),   S_c = max over the seen keys j of block c of s_j,
// -inf for a block without one; a NaN counts as -inf.
//
// Keys on M. A tile is 128 keys (A, 128 bytes each) against the heads of a group of neighbouring tokens
// of one sequence (B, up to NB rows of 128 bytes): four E4M3 MMAs of K = 32, exact products, float32
// sums in tensor memory, a key in each lane and a head in each column. So the sum over heads stays in a
// thread, w_h is the same for all lanes, and only the maximum over a block's keys crosses lanes. A
// token's heads start at a multiple of 16 columns; the columns between hold whatever follows in memory
// and are never read.
//
// Work is cut into units of one group x `unit_blocks` blocks; persistent CTAs, one per SM, take them in
// turn, all groups of one stretch of the context before the next, so that groups of a sequence find
// its keys in L2. A group's number says which sequence it belongs to: sequence b's groups start at
// cu_q[b] / TG + b (TG tokens to a group), which leaves room enough for each, and a lane finds its
// unit's by bisection.
//
// Roles (320 threads): warp 0 resolves units, fills blocks that no token sees, and loads queries, weights,
// keys (TMA boxes from the page table) and their scales; warp 1 issues the MMAs; warps 2-5 and 6-9 take
// the tiles in turn, each with an accumulator of its own. The maxima of a unit's blocks gather in shared
// memory. Every wait is bounded; a stall sets the error word, and the CTA drains and leaves.
#include "mla_index.h"
#include "mla_ptx.cuh"
#include "mla_ragged.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kISThreads = 320;
constexpr int kISKeys = 128;                      // keys of a tile
constexpr int kISSlotBytes = kISKeys * kDIndex;   // 16 KB
constexpr int kISSlots = 7;
constexpr int kISBest = 2048;                     // (token, block) maxima of a unit
constexpr int kISMaxTokens = 16;                  // 256 columns / 16

template <int NB>
constexpr int is_smem_bytes() {
  return 1024 + 2 * NB * kDIndex + kISSlots * (kISSlotBytes + kISKeys * 4) + 2 * kISBest * 4 + 2 * NB * 4;
}

// an order-preserving code of a float, so that maxima can be taken as integers
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }
constexpr int kLowest = (int)0x807FFFFFu;         // ordered(-inf)

// max(0, x) that keeps a NaN
__device__ __forceinline__ float positive(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}
// (a, b) += (x, y) * (u, v)
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float u, float v) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%0, %1};\n\t"
      "fma.rn.f32x2 r, p, q, r;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "+f"(a), "+f"(b) : "f"(x), "f"(y), "f"(u), "f"(v));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// bytes (a multiple of 16) from global to this CTA's shared memory, counted on `bar`
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
}

// A unit as the producer announces it.
struct UnitInfo {
  int t0, ntok;          // its tokens; ntok = 0: no more units
  int k0, tiles;         // first key, tiles of 128 keys
  int c0, blocks;        // first column of the scores, columns to be written
  int seen[kISMaxTokens];
};

__device__ uint32_t g_unreported;                 // error bits of calls without an error word

}  // namespace

template <int NB>
__global__ void __launch_bounds__(kISThreads, 1) index_scores_kernel(const __grid_constant__ IndexScoreArgs a) {
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ __align__(8) uint64_t bar_kfull[kISSlots], bar_kempty[kISSlots], bar_qfull[2], bar_qempty[2], bar_tfull[2],
      bar_tempty[2], bar_unit, bar_drain, bar_never;
  __shared__ UnitInfo info_s[2];
  __shared__ uint32_t tmem_base_s, abort_s;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(dsmem_raw);
  const uint32_t sQ = (raw + 1023u) & ~1023u, sK = sQ + 2 * NB * kDIndex;
  uint8_t* gQ = dsmem_raw + (sQ - raw);
  float* gS = reinterpret_cast<float*>(gQ + 2 * NB * kDIndex + kISSlots * kISSlotBytes);   // key scales
  const uint32_t sS = sK + kISSlots * kISSlotBytes;
  int* best = reinterpret_cast<int*>(gS + kISSlots * kISKeys);                             // [2][kISBest]
  float* gW = reinterpret_cast<float*>(best + 2 * kISBest);                                // [2][NB]
  const uint32_t b_kfull = smem_u32(bar_kfull), b_kempty = smem_u32(bar_kempty);
  const uint32_t b_qfull = smem_u32(bar_qfull), b_qempty = smem_u32(bar_qempty);
  const uint32_t b_tfull = smem_u32(bar_tfull), b_tempty = smem_u32(bar_tempty);
  const uint32_t b_unit = smem_u32(&bar_unit), b_drain = smem_u32(&bar_drain), b_never = smem_u32(&bar_never);
  volatile uint32_t* abort_flag = &abort_s;
  uint32_t* err = a.err != nullptr ? a.err : &g_unreported;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kISSlots; ++i) {
      mbar_init(b_kfull + 8 * i, 1);
      mbar_init(b_kempty + 8 * i, 1 + 4);     // the MMAs, and the warps that have read the scales
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_qfull + 8 * i, 1);
      mbar_init(b_qempty + 8 * i, 1 + 8);     // the MMAs, and the warps that are done with the unit
      mbar_init(b_tfull + 8 * i, 1);
      mbar_init(b_tempty + 8 * i, 4);
    }
    mbar_init(b_unit, 8);
    mbar_init(b_drain, 1);
    mbar_init(b_never, 1);
    abort_s = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_base_s), 2 * NB);
  for (int i = threadIdx.x; i < 2 * kISBest; i += kISThreads) best[i] = kLowest;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  griddep_wait();
  griddep_launch_dependents();
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns));
  };
  const int TG = a.TG, Hp = a.Hp;

  if (warp == 0) {
    // ---------------------------------------------------------------------- units, queries, keys
    const bool el = elect_one();
    const int per = kISKeys / a.box_rows;               // boxes of a tile: lane i issues box i
    uint32_t slot = 0, ph = 1, nu = 0, filled = 0;
    bool ok = true;
    const int64_t total = (int64_t)a.slots * a.chunks;
    for (int64_t base = blockIdx.x; base < total && ok; base += 32 * (int64_t)gridDim.x) {
      // 32 units at a time, one to a lane
      const int64_t u = base + (int64_t)lane * gridDim.x;
      int b = 0, t0 = 0, ntok = 0, k0 = 0, c0 = 0, last = 0, start = 0, end = 0, L = 0;
      if (u < total) {
        const int chunk = (int)(u / a.slots), g = (int)(u - (int64_t)chunk * a.slots);
        int lo = 0, hi = a.B;                           // the last b with cu_q[b] / TG + b <= g
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (a.cu_q[mid] / TG + mid <= g) lo = mid;
          else hi = mid;
        }
        b = lo;
        start = max(0, a.cu_q[b]);
        end = min(a.T, a.cu_q[b + 1]);
        const int64_t first = (int64_t)start + (int64_t)(g - (start / TG + b)) * TG;
        if (g >= start / TG + b && first < end) {
          t0 = (int)first;
          ntok = min(TG, end - t0);
          L = max(0, min(a.seq_lens[b], a.max_len));
          c0 = chunk * a.unit_blocks;
          k0 = c0 * a.block;
          last = min(keys_seen(t0 + ntok - 1, start, end, L, a.causal), k0 + a.unit_blocks * a.block);
        }
      }
      const uint32_t any = __ballot_sync(0xffffffffu, ntok > 0);
      for (uint32_t m = any; m != 0 && ok; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int ub = __shfl_sync(0xffffffffu, b, src), ut0 = __shfl_sync(0xffffffffu, t0, src);
        const int un = __shfl_sync(0xffffffffu, ntok, src), uk0 = __shfl_sync(0xffffffffu, k0, src);
        const int uc0 = __shfl_sync(0xffffffffu, c0, src), ulast = __shfl_sync(0xffffffffu, last, src);
        const int ustart = __shfl_sync(0xffffffffu, start, src), uend = __shfl_sync(0xffffffffu, end, src);
        const int uL = __shfl_sync(0xffffffffu, L, src);
        const int blocks = min(a.unit_blocks, a.C - uc0);
        if (ulast <= uk0) {                             // no token sees these blocks
          for (int i = 0; i < un; ++i)
            for (int c = lane; c < blocks; c += 32) a.out[(int64_t)(ut0 + i) * a.C + uc0 + c] = -INFINITY;
          continue;
        }
        const int tiles = (ulast - uk0 + kISKeys - 1) / kISKeys;
        const uint32_t qb = nu & 1;
        ok = wait(b_qempty + 8 * qb, ((nu >> 1) & 1) ^ 1);
        if (!ok) break;
        UnitInfo& I = info_s[qb];
        if (lane == 0) {
          I.t0 = ut0;
          I.ntok = un;
          I.k0 = uk0;
          I.tiles = tiles;
          I.c0 = uc0;
          I.blocks = blocks;
        }
        if (lane < un) I.seen[lane] = keys_seen(ut0 + lane, ustart, uend, uL, a.causal);
        for (int i = lane; i < un * a.H; i += 32) gW[qb * NB + (i / a.H) * Hp + i % a.H] = a.w[(int64_t)ut0 * a.H + i];
        __syncwarp();
        const int qboxes = un * (Hp / 16);
        if (el) mbar_arrive_expect_tx(b_qfull + 8 * qb, (uint32_t)qboxes * 16 * kDIndex);
        __syncwarp();
        for (int i = lane; i < qboxes; i += 32)
          tma_load_2d(sQ + qb * NB * kDIndex + i * 16 * kDIndex, &a.tm_q, b_qfull + 8 * qb, 0,
                      (ut0 + i / (Hp / 16)) * a.H + (i % (Hp / 16)) * 16);
        ++nu;
        // a lane's boxes of the unit: their pages one tile ahead
        const int32_t* pages = a.block_table + (int64_t)ub * a.MB;
        auto row_of = [&](int tile) -> int {
          const int tok = uk0 + tile * kISKeys + lane * a.box_rows;
          if (lane >= per || tok >= ulast) return -1;
          const int page = tok / a.P, in = tok - page * a.P;
          int pg = __ldg(pages + page);
          if (pg < 0 || pg >= a.num_pages) {
            atomicOr(err, MLA_DEVERR_BLOCK_TABLE);
            pg = 0;
          }
          return pg * a.P + in;
        };
        int row = row_of(0);
        for (int tile = 0; tile < tiles; ++tile) {
          const int next = tile + 1 < tiles ? row_of(tile + 1) : -1;
          ok = wait(b_kempty + 8 * slot, ph);
          if (!ok) break;
          const int valid = __popc(__ballot_sync(0xffffffffu, row >= 0));
          const uint32_t bar = b_kfull + 8 * slot;
          if (el) mbar_arrive_expect_tx(bar, kISSlotBytes + (uint32_t)(valid * a.box_rows * 4));
          __syncwarp();
          if (lane < per) {
            // a box past the keys starts at the end of the pool and reads zeros
            tma_load_2d(sK + slot * kISSlotBytes + lane * a.box_rows * kDIndex, &a.tm_k, bar, 0,
                        row >= 0 ? row : a.total_rows);
            if (row >= 0)
              bulk_load(sS + (slot * kISKeys + lane * a.box_rows) * 4, a.scale + row, (uint32_t)a.box_rows * 4, bar);
          }
          row = next;
          ++filled;
          if (++slot == kISSlots) { slot = 0; ph ^= 1; }
        }
      }
    }
    // the end of the units
    if (ok) {
      const uint32_t qb = nu & 1;
      ok = wait(b_qempty + 8 * qb, ((nu >> 1) & 1) ^ 1);
      if (ok) {
        if (lane == 0) info_s[qb].ntok = 0;
        __syncwarp();
        if (el) mbar_arrive(b_qfull + 8 * qb);
      }
    }
    if (!ok) {
      // copies in flight land before the CTA leaves: the last fill of each slot
      volatile uint32_t none = 0u;
      if (lane == 0) {
        for (uint32_t f = filled > kISSlots ? filled - kISSlots : 0; f < filled; ++f)
          mbar_wait(b_kfull + 8 * (f % kISSlots), (f / kISSlots) & 1, &none, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
        for (uint32_t k = nu >= 2 ? nu - 2 : 0; k < nu; ++k)
          mbar_wait(b_qfull + 8 * (k & 1), (k >> 1) & 1, &none, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------------------------- MMAs
    const bool el = elect_one();
    uint32_t slot = 0, ph = 0, nt = 0;
    bool ok = true;
    for (uint32_t nu = 0; ok; ++nu) {
      const uint32_t qb = nu & 1;
      ok = wait(b_qfull + 8 * qb, (nu >> 1) & 1);
      if (!ok) break;
      const int ntok = info_s[qb].ntok, tiles = info_s[qb].tiles;
      if (ntok == 0) break;
      const uint32_t idesc = make_idesc(128, (uint32_t)(ntok * Hp), 0, 0, 0);
      const uint64_t qd = make_sdesc(sQ + qb * NB * kDIndex, 16, 1024, kSwizzle128);
      for (int tile = 0; tile < tiles; ++tile, ++nt) {
        const uint32_t st = nt & 1;
        ok = wait(b_tempty + 8 * st, ((nt >> 1) & 1) ^ 1) && wait(b_kfull + 8 * slot, ph);
        if (!ok) break;
        tc_fence_after();
        if (el) {
          const uint64_t kd = make_sdesc(sK + slot * kISSlotBytes, 16, 1024, kSwizzle128);
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_f8(tmem + st * NB, kd + 2 * k, qd + 2 * k, idesc, k > 0);
          umma_commit(b_kempty + 8 * slot);
          umma_commit(b_tfull + 8 * st);
          if (tile + 1 == tiles) umma_commit(b_qempty + 8 * qb);
        }
        __syncwarp();
        if (++slot == kISSlots) { slot = 0; ph ^= 1; }
      }
    }
    if (!ok) {
      // the MMAs issued so far complete before tensor memory is freed
      volatile uint32_t none = 0u;
      if (el) {
        umma_commit(b_drain);
        mbar_wait(b_drain, 0, &none, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- sums over heads, maxima over keys
    const uint32_t wg = warp >= 6 ? 1u : 0u;
    const int quad = warp & 3;                          // tensor-memory lanes 32 quad ..
    const int et = threadIdx.x - 64;                    // thread of the 256
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + wg * NB;
    // errors that only the device can see
    for (int b = blockIdx.x * 256 + et; b < a.B; b += gridDim.x * 256) {
      const uint32_t bad = ragged_errors(a.cu_q, a.seq_lens, b, a.T, a.max_len);
      if (bad) atomicOr(err, bad);
    }
    uint32_t slot = 0, ph = 0, nt = 0;
    bool ok = !(a.test_stall && !wait(b_never, 0));
    const bool whole = a.block % 32 == 0;               // a warp's keys lie in one block
    const int H = a.H;
    for (uint32_t nu = 0; ok; ++nu) {
      const uint32_t qb = nu & 1;
      ok = wait(b_qfull + 8 * qb, (nu >> 1) & 1);
      if (!ok) break;
      const UnitInfo& I = info_s[qb];
      const int ntok = I.ntok, tiles = I.tiles;
      if (ntok == 0) break;
      int* mine = best + qb * kISBest;
      for (int tile = 0; tile < tiles; ++tile, ++nt) {
        const uint32_t my_slot = slot, my_ph = ph;
        if (++slot == kISSlots) { slot = 0; ph ^= 1; }
        if ((nt & 1) != wg) continue;
        ok = wait(b_tfull + 8 * wg, (nt >> 1) & 1) && wait(b_kfull + 8 * my_slot, my_ph);
        if (!ok) break;
        tc_fence_after();
        const float ks = gS[my_slot * kISKeys + quad * 32 + lane];
        __syncwarp();
        if (lane == 0) mbar_arrive(b_kempty + 8 * my_slot);
        const int in = tile * kISKeys + quad * 32 + lane;     // key within the unit
        const int key = I.k0 + in;
        const int block = (whole ? in - lane : in) / a.block;
        int keep = kLowest;
        for (int i = 0; i < ntok; ++i) {
          const float* w = gW + qb * NB + i * Hp;
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
          int c = 0;
          for (; c + 32 <= H; c += 32) {
            float v[32];
            tmem_ld32(lane_base + i * Hp + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 x = *reinterpret_cast<const float4*>(w + c + k);
              fma2(s0, s1, positive(v[k]), positive(v[k + 1]), x.x, x.y);
              fma2(s2, s3, positive(v[k + 2]), positive(v[k + 3]), x.z, x.w);
            }
          }
          for (; c < H; c += 16) {
            float v[16];
            tmem_ld16(lane_base + i * Hp + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c + k < H) s0 = fmaf(positive(v[k]), w[c + k], s0);
          }
          float s = ((s0 + s1) + (s2 + s3)) * ks;
          s = key < I.seen[i] && s > -INFINITY ? s : -INFINITY;
          if (whole) {
            const int m = __reduce_max_sync(0xffffffffu, ordered(s));
            if (lane == i) keep = m;
          } else {
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
            if ((lane & 7) == 0) atomicMax(mine + i * a.unit_blocks + block, ordered(s));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_tempty + 8 * wg);
        if (whole && lane < ntok) atomicMax(mine + lane * a.unit_blocks + block, keep);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_unit);               // all eight warps' maxima are in
      ok = wait(b_unit, nu & 1);
      if (!ok) break;
      const int n = ntok * a.unit_blocks;
      for (int x = et; x < n; x += 256) {
        const int i = x / a.unit_blocks, c = x - i * a.unit_blocks;
        if (c < I.blocks) a.out[(int64_t)(I.t0 + i) * a.C + I.c0 + c] = from_ordered(mine[x]);
        mine[x] = kLowest;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_qempty + 8 * qb);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * NB);
}

// Columns of the accumulators: a decode step's groups are one token, whose heads take 64 or 128; with
// two tokens or more to a sequence on average, up to 256 columns of them share each key tile.
int index_scores_columns(int T, int B, int H) { return T >= 2 * (int64_t)B ? 256 : H <= 64 ? 64 : 128; }

cudaError_t launch_index_scores(IndexScoreArgs a, int columns, int num_sms, cudaStream_t s) {
  a.Hp = (a.H + 15) / 16 * 16;
  a.TG = columns / a.Hp;
  if (columns < 256) a.TG = 1;
  if (a.TG > kISMaxTokens) a.TG = kISMaxTokens;
  a.slots = a.T / a.TG + a.B;
  // a unit: whole blocks and whole tiles, about eight units to a CTA, 512 to 8192 keys
  int lcm = a.block;
  while (lcm % kISKeys != 0) lcm += a.block;
  const int64_t groups = (a.T + a.TG - 1) / a.TG;
  int64_t keys = groups * a.max_len / (8 * (int64_t)num_sms);
  keys = keys < 512 ? 512 : keys > (columns < 256 ? 1024 : 8192) ? (columns < 256 ? 1024 : 8192) : keys;
  int64_t m = keys / lcm;
  const int64_t most = kISBest / ((int64_t)a.TG * (lcm / a.block));
  m = m > most ? most : m;
  if (m < 1) m = 1;
  a.unit_blocks = (int)(m * (lcm / a.block));
  a.chunks = (a.C + a.unit_blocks - 1) / a.unit_blocks;
  const int64_t total = (int64_t)a.slots * a.chunks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(total < num_sms ? total : num_sms));
  cfg.blockDim = dim3(kISThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto* kernel, int smem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  if (columns == 64) return go(index_scores_kernel<64>, is_smem_bytes<64>());
  if (columns == 128) return go(index_scores_kernel<128>, is_smem_bytes<128>());
  return go(index_scores_kernel<256>, is_smem_bytes<256>());
}

}  // namespace mla
