// mla_index_scores.cu — scores of the blocks of a ragged batch's contexts (sm_103a, tcgen05).
//
// For token t, key j it sees and block c of `block` keys:
//   s_j = scale_j sum_h w_h max(0, q_h . k_j),   S_c = max over the seen keys j of block c of s_j,
// -inf for a block without one; a NaN counts as -inf.
//
// Keys on M. A tile is 128 keys (A, 128 bytes each) against the heads of a few tokens of one sequence
// (B, up to 128 rows of 128 bytes): four E4M3 MMAs of K = 32, exact products, float32 sums in tensor
// memory, a key in each lane and a head in each column. So the sum over heads stays in a thread, w_h is the
// same for all lanes, and only the maximum over a block's keys crosses lanes. A token takes 16, 32, 64 or
// 128 columns; those without a head have queries and weights of zero.
//
// Work is cut into units of one group of up to TG neighbouring tokens x some `unit_blocks` blocks, as far as the
// context goes; persistent CTAs, one per SM, take them in turn. Units are numbered by sequence and, within
// one, all groups of a stretch of the context before the next, so that groups of a sequence find its keys
// in L2. Each CTA counts them itself, 512 sequences at a time, and a lane finds its unit's sequence by
// bisection: 32 units at once. A group is up to four sub-groups of 128 columns, which share each key tile
// in shared memory.
//
// Roles (640 threads): warp 0 counts units, loads their queries and weights, and writes their scores;
// warp 3 loads keys (TMA boxes from the page table) and their scales; warps 1 and 2 issue the MMAs, each into a
// pair of accumulators of 128 columns: two sub-groups of a tile, or two tiles of one; four warpgroups take
// an accumulator each. The maxima of a unit's blocks gather in shared memory. Every wait is bounded; a stall
// sets the error word, and the CTA drains and leaves.
//
// What bounds it. Many tokens: the sums. 32 columns of 128 keys take a scheduler's four warps 58 instructions and
// 90 clocks each at best (a loop apart: 73 without max, 58 without the tensor-memory loads), the MMAs 64; with
// maxima, waits and bookkeeping it is about 97 instructions and 142 clocks. 2048 tokens x 64 heads over 24 K keys
// 400 us (2.1 PFLOP/s of E4M3; 44% of tensor cycles), with 16 heads 129 (219 while the warp that loads queries and
// writes scores went through a unit's tokens one by one, a box for each). On the way there: one issuing warp held
// back everything (546 us for four warpgroups, its products of 128 columns take it 570 clocks), two of them 490,
// products of 256 columns 457; a chunk more of double buffering or a quarter of max on the FMA pipe, 3%.
// Few tokens: latency and the loading warp. 121 sequences x 4 K keys 17.2 us for 65 MB (21.2 where they come from
// DRAM), of which 6 us pass before the first product and after the last; with one warp for units and keys 32, with
// keys' scales as bulk copies 24 (each takes the warp about 95 clocks to issue, like a key box), tile by tile 21.5,
// with integer divisions where a unit's pages are looked up 18.4.
#include <type_traits>
#include "mla_index.h"
#include "mla_ptx.cuh"
#include "mla_ragged.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kISWarps = 16;                      // four warpgroups, two to a pair of accumulators
constexpr int kISIssuers = 2;                     // issuing warps, one to a pair of accumulators
constexpr int kISFirst = 2 + kISIssuers;          // first warp of the warpgroups
constexpr int kISThreads = 32 * (kISFirst + kISWarps);
constexpr int kISColumns = 128;                   // of an accumulator
constexpr int kISTmem = 2 * kISIssuers * kISColumns;
constexpr int kISKeys = 128;                      // keys of a tile
constexpr int kISSlotBytes = kISKeys * kDIndex;   // 16 KB
constexpr int kISMaxSlots = 12;
constexpr int kISTogether = 8;                    // tiles whose loads are issued at once, where there are slots for them
// Key scales have a ring of their own, read later than the keys. A slot of it is filled for tile t + 16
// once the keys of tile t + 4 or a later one have been given back by both issuing warps. A product covers
// two tiles at most and the two pairs of accumulators alternate, so by then the warp that issued tile t's
// product has issued its next one, which waited until tile t's had been read.
constexpr int kISScales = 16;
constexpr uint32_t kISFirstWaitNs = 20000;        // a wait's first, sleeping look
constexpr int kISBest = 1024;                     // (token, block) maxima of a unit, at most
constexpr int kISMaxUnits = 4;                    // units whose queries are in shared memory
constexpr int kISMaxTokens = 32;                  // of a group: 512 columns / 16
constexpr int kISSeqs = 512;                      // sequences whose units are counted at a time
constexpr int kISSmem = 216 * 1024;               // dynamic
// all but the key tiles: queries, scales, maxima, weights
constexpr int is_fixed_bytes(int units, int q_rows, int maxima) {
  return 1024 + kISScales * kISKeys * 4 + units * (q_rows * kDIndex + maxima * 4 + q_rows * 4);
}
constexpr int is_key_slots(int units, int q_rows, int maxima) {
  return (kISSmem - is_fixed_bytes(units, q_rows, maxima)) / kISSlotBytes;
}
constexpr int kISMaxRows = 2 * kISIssuers * kISColumns;   // of a query buffer: four sub-groups
constexpr int kISManyRows = kISMaxRows / 2;               // up to which there are kISMaxUnits buffers, else 2
static_assert(is_key_slots(2, kISMaxRows, kISBest) >= 2 && is_key_slots(kISMaxUnits, kISManyRows, kISBest) >= 2,
              "a product of one sub-group takes two tiles of keys at once");
static_assert(kISMaxTokens * (kISKeys / 8) <= kISBest, "the smallest unit of a full group");
static_assert(kISScales >= kISMaxSlots + 4, "scales are read until four tiles later");
static_assert(kISTogether <= 32, "a lane for each tile");

// an order-preserving code of a float, so that maxima can be taken as integers
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }
constexpr int kLowest = (int)0x807FFFFFu;         // ordered(-inf)

// Two values to an instruction: acc = w max(0, (x, y)) + (first ? 0 : acc), NaN kept. Volatile, so that it stays
// behind the wait for the tensor-memory load that brings x and y.
template <bool kFirst>
__device__ __forceinline__ void add_positive2(uint64_t& acc, float x, float y, uint64_t w) {
  if (kFirst)
    asm volatile("{\n\t.reg .f32 a, b;\n\t.reg .b64 p;\n\tmax.NaN.f32 a, %1, 0f00000000;\n\t"
                 "max.NaN.f32 b, %2, 0f00000000;\n\tmov.b64 p, {a, b};\n\tmul.rn.f32x2 %0, p, %3;\n\t}"
                 : "=l"(acc) : "f"(x), "f"(y), "l"(w));
  else
    asm volatile("{\n\t.reg .f32 a, b;\n\t.reg .b64 p;\n\tmax.NaN.f32 a, %1, 0f00000000;\n\t"
                 "max.NaN.f32 b, %2, 0f00000000;\n\tmov.b64 p, {a, b};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
                 : "+l"(acc) : "f"(x), "f"(y), "l"(w));
}
// The same with x + |x| = 2 max(0, x) in its place, on the FMA pipe instead of the ALU: these sums are halved at the
// end, so they overflow from 2^127 on. (Half of it as a further operand costs an instruction for each pair.)
template <bool kFirst>
__device__ __forceinline__ void add_positive2_twice(uint64_t& acc, float x, float y, uint64_t w) {
  if (kFirst)
    asm volatile("{\n\t.reg .f32 a, b;\n\t.reg .b64 p;\n\tabs.f32 a, %1;\n\tabs.f32 b, %2;\n\tadd.rn.f32 a, a, %1;\n\t"
                 "add.rn.f32 b, b, %2;\n\tmov.b64 p, {a, b};\n\tmul.rn.f32x2 %0, p, %3;\n\t}"
                 : "=l"(acc) : "f"(x), "f"(y), "l"(w));
  else
    asm volatile("{\n\t.reg .f32 a, b;\n\t.reg .b64 p;\n\tabs.f32 a, %1;\n\tabs.f32 b, %2;\n\tadd.rn.f32 a, a, %1;\n\t"
                 "add.rn.f32 b, b, %2;\n\tmov.b64 p, {a, b};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
                 : "+l"(acc) : "f"(x), "f"(y), "l"(w));
}
// three pairs, and half of the fourth
__device__ __forceinline__ float sum8(const uint64_t* s) {
  float r;
  asm("{\n\t.reg .b64 a, b;\n\t.reg .f32 x, y, u, v;\n\tadd.rn.f32x2 a, %1, %2;\n\tadd.rn.f32x2 a, a, %3;\n\t"
      "mov.b64 {x, y}, a;\n\tmov.b64 {u, v}, %4;\n\tadd.rn.f32 x, x, y;\n\tadd.rn.f32 u, u, v;\n\t"
      "fma.rn.f32 %0, u, 0f3F000000, x;\n\t}"
      : "=f"(r) : "l"(s[0]), "l"(s[1]), "l"(s[2]), "l"(s[3]));
  return r;
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
// 16 bytes from global to this CTA's shared memory, asynchronously; and this thread's arrival on `bar` once
// its copies so far have landed (counted as pending from the start)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared::cta.global [%0], [%1], 16;" :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                 "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                 "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// the largest of the warp's values, NaN aside (NaN if all are)
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// CS heads of a token, its first ones or further ones, in four pairs of sums for short chains. max runs
// on the ALU at half the rate of the FMA pipe: a quarter of the heads takes the other form.
template <int CS, bool kFirst>
__device__ __forceinline__ void add_heads(const float* v, const float* w, uint64_t* s) {
#pragma unroll
  for (int k = 0; k < CS; k += 8) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + k), y = *reinterpret_cast<const ulonglong2*>(w + k + 4);
    if (kFirst && k == 0) {
      add_positive2<true>(s[0], v[k], v[k + 1], x.x);
      add_positive2<true>(s[1], v[k + 2], v[k + 3], x.y);
      add_positive2<true>(s[2], v[k + 4], v[k + 5], y.x);
      add_positive2_twice<true>(s[3], v[k + 6], v[k + 7], y.y);
    } else {
      add_positive2<false>(s[0], v[k], v[k + 1], x.x);
      add_positive2<false>(s[1], v[k + 2], v[k + 3], x.y);
      add_positive2<false>(s[2], v[k + 4], v[k + 5], y.x);
      add_positive2_twice<false>(s[3], v[k + 6], v[k + 7], y.y);
    }
  }
}
// e / d of a small e, with by = (2^32 - 1) / d rounded down: (e + 1) by falls short of (e + 1) 2^32 / d by less than 2^32 / d
__device__ __forceinline__ int quotient(int e, uint32_t by) { return (int)__umulhi((uint32_t)e + 1u, by); }

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<uint64_t>(p)));
}

// The rest of a wait that was not over at the first look, out of line.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, uint32_t abort_s, uint32_t* err, uint64_t limit_ns) {
  volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(__cvta_shared_to_generic(abort_s));
  return mbar_wait(bar, parity, flag, err, MLA_DEVERR_TIMEOUT, limit_ns);
}

// A unit as the producer announces it.
struct UnitInfo {
  int t0, ntok, seq;     // its tokens and their sequence; ntok = 0: no more units
  int k0, last, tiles;   // first key, end of the keys that a token sees, tiles of 128 keys
  int c0, blocks, rest;  // first column of the scores, columns with maxima and those of -inf behind them
  int seen[kISMaxTokens];
};

__device__ uint32_t g_unreported;                 // error bits of calls without an error word

}  // namespace

// A token's heads take PT chunks of CS columns, 16, 32, 64 or 128 (at least as many as heads). kWhole: blocks
// are a multiple of 32 keys, so that a warp's keys lie in one.
template <int CS, int PT, bool kWhole>
__global__ void __launch_bounds__(kISThreads, 1) index_scores_kernel(const __grid_constant__ IndexScoreArgs a) {
  constexpr int Hp = CS * PT, kFull = kISColumns / Hp;   // columns of a token, tokens of an accumulator
  constexpr int kAtOnce = 32 / CS;                  // tokens of a load from tensor memory
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ __align__(8) uint64_t bar_kfull[kISMaxSlots], bar_kempty[kISMaxSlots], bar_info[kISMaxUnits],
      bar_qfull[kISMaxUnits], bar_qempty[kISMaxUnits], bar_tfull[kISIssuers], bar_tempty[kISIssuers], bar_drain[kISIssuers], bar_never;
  __shared__ UnitInfo info_s[kISMaxUnits];
  __shared__ int cu_s[kISSeqs + 1], len_s[kISSeqs];
  __shared__ uint32_t first_s[kISSeqs + 1];         // a sequence's first unit
  __shared__ uint32_t tmem_base_s, abort_s;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int S = a.key_slots, q_rows = a.q_rows, units = a.units, maxima = a.TG * a.unit_blocks;
  const uint32_t raw = smem_u32(dsmem_raw);
  const uint32_t sQ = (raw + 1023u) & ~1023u, sK = sQ + units * q_rows * kDIndex;
  const uint32_t sS = sK + S * kISSlotBytes;
  float* gS = reinterpret_cast<float*>(dsmem_raw + (sS - raw));       // key scales
  float* gW = gS + kISScales * kISKeys;                               // [units][q_rows]
  int* best = reinterpret_cast<int*>(gW + units * q_rows);            // [units][maxima]
  const uint32_t b_kfull = smem_u32(bar_kfull), b_kempty = smem_u32(bar_kempty);
  const uint32_t b_info = smem_u32(bar_info), b_qfull = smem_u32(bar_qfull), b_qempty = smem_u32(bar_qempty);
  const uint32_t b_tfull = smem_u32(bar_tfull), b_tempty = smem_u32(bar_tempty);
  const uint32_t b_drain = smem_u32(bar_drain), b_never = smem_u32(&bar_never);
  uint32_t* err = a.err != nullptr ? a.err : &g_unreported;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kISMaxSlots; ++i) {
      mbar_init(b_kfull + 8 * i, 1 + 32);           // the keys, and the loading warp's scales
      mbar_init(b_kempty + 8 * i, kISIssuers);
    }
    for (int i = 0; i < kISMaxUnits; ++i) {
      mbar_init(b_info + 8 * i, 1);
      mbar_init(b_qfull + 8 * i, 1);
      mbar_init(b_qempty + 8 * i, kISIssuers + kISWarps);   // the MMAs, and the warps that are done with the unit
    }
    for (int i = 0; i < kISIssuers; ++i) {
      mbar_init(b_tfull + 8 * i, 2);               // the MMAs, and the issuing thread, which saw the scales land
      mbar_init(b_tempty + 8 * i, 8);
      mbar_init(b_drain + 8 * i, 1);
    }
    mbar_init(b_never, 1);
    abort_s = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_base_s), kISTmem);
  for (int i = threadIdx.x; i < units * maxima; i += kISThreads) best[i] = kLowest;
  // Where heads fill a token's columns, a unit's weights come by one bulk copy. Else by loads and ordinary stores,
  // and columns without a head keep the zeros written here (with bulk copies there are none: nothing would order these
  // stores, of the generic proxy, before the copy's, of the async proxy).
  const bool bulk_weights = a.H == Hp && (reinterpret_cast<uintptr_t>(a.w) & 15) == 0;
  if (!bulk_weights)
    for (int i = threadIdx.x; i < units * q_rows; i += kISThreads) gW[i] = 0.f;
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, kISFirstWaitNs) ||
                                       wait_longer(bar, parity, smem_u32(&abort_s), err, a.wait_limit_ns));
  };
  constexpr int sub_tokens = kFull;
  const int TG = a.TG;

  if (warp == 0) {
    // ---------------------------------------------------------------------- units and their queries
    const bool el = elect_one();
    uint32_t ub = 0, uph = 1, nu = 0;                   // the unit's buffer and the parity of its barriers, units so far
    bool ok = true;
    int unit_blocks = a.usual_blocks, unit_keys = unit_blocks * a.block;
    // waits until a buffer's last unit is done, and writes its scores
    auto finish_unit = [&](uint32_t buffer, uint32_t parity, bool used) -> bool {
      if (!wait(b_qempty + 8 * buffer, parity)) return false;
      if (!used) return true;
      const UnitInfo& I = info_s[buffer];
      int* from = best + buffer * maxima;
      float* to = a.out + (int64_t)I.t0 * a.C + I.c0;
      const int n = I.ntok * a.unit_blocks, blocks = I.blocks, rest = I.rest;
#pragma unroll 1                                        // (shorter code beats more loads at once, 403 us against 400)
      for (int e = lane; e < n; e += 32) {              // of all tokens at once
        const int i = quotient(e, a.by_blocks), c = e - i * a.unit_blocks;
        if (c < blocks) to[(int64_t)i * a.C + c] = from_ordered(from[e]);
        from[e] = kLowest;
      }
      for (int i = 0; rest > 0 && i < I.ntok; ++i)
        for (int c = lane; c < rest; c += 32) to[(int64_t)i * a.C + blocks + c] = -INFINITY;
      __syncwarp();
      return true;
    };
    int64_t next = blockIdx.x, counted = 0;             // this CTA's next unit; units of the sequences before
    for (int b0 = 0; b0 < a.B && ok; b0 += kISSeqs) {
      // units of up to 512 sequences
      const int nb = min(a.B - b0, kISSeqs);
      for (int i = lane; i <= nb; i += 32) cu_s[i] = a.cu_q[b0 + i];
      for (int i = lane; i < nb; i += 32) len_s[i] = max(0, min(a.seq_lens[b0 + i], a.max_len));
      __syncwarp();
      uint32_t units_before = 0;
      if (a.choose) {
        // Few units: of a size that makes few rounds of short ones. A unit costs about as much as its tiles
        // and 1.5 more; lane l looks at l + 1 steps.
        uint32_t tiles = 0, groups = 0;
        for (int i = lane; i < nb; i += 32) {
          const uint32_t g = (uint32_t)(max(0, cu_s[i + 1] - cu_s[i]) + TG - 1) >> a.tg_log2;
          tiles += g * (uint32_t)((len_s[i] + kISKeys - 1) / kISKeys);
          groups += g;
        }
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        groups = __reduce_add_sync(0xffffffffu, groups);
        const float m = (float)((lane + 1) * a.step_tiles);
        const float units = __fdividef((float)tiles + 0.5f * (float)groups * (m - 1.f), m);
        const float cost = fminf(ceilf(units * a.by_grid) * (m + 1.5f) * 64.f, 1e8f);
        const bool fits = (lane + 1) * a.step_blocks <= a.unit_blocks;
        const uint32_t best = __reduce_min_sync(0xffffffffu, fits ? (uint32_t)cost << 5 | (uint32_t)lane : 0xFFFFFFFFu);
        unit_blocks = (int)((best & 31) + 1) * a.step_blocks;
        unit_keys = unit_blocks * a.block;
      }
      bool bad = false;
      for (int i0 = 0; i0 < nb; i0 += 32) {
        uint32_t mine = 0;
        if (i0 + lane < nb) {
          const int n = cu_s[i0 + lane + 1] - cu_s[i0 + lane];
          bad |= cu_s[i0 + lane] < 0 || n < 0 || cu_s[i0 + lane + 1] > a.T;
          // (a sequence without keys has a unit that sees none)
          if (n > 0) mine = (uint32_t)((n + TG - 1) >> a.tg_log2) * (uint32_t)max(1, (len_s[i0 + lane] + unit_keys - 1) / unit_keys);
        }
        uint32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (i0 + lane < nb) first_s[i0 + lane] = units_before + x - mine;
        units_before += __shfl_sync(0xffffffffu, x, 31);
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, bad)) break;          // offsets that do not ascend: no scores from here on
      const int64_t end_units = counted + units_before;
      for (; next < end_units && ok; next += 32 * (int64_t)gridDim.x) {
        // 32 units at a time, one to a lane
        const int64_t u = next + (int64_t)lane * gridDim.x;
        int b = 0, t0 = 0, ntok = 0, chunk = 0, start = 0, end = 0, L = 0;
        if (u < end_units) {
          const uint32_t r = (uint32_t)(u - counted);
          int hi = nb;                                  // the last sequence whose first unit is at most r
          while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (first_s[mid] <= r) b = mid;
            else hi = mid;
          }
          start = cu_s[b];
          end = cu_s[b + 1];
          L = len_s[b];
          const uint32_t groups = (uint32_t)((end - start + TG - 1) >> a.tg_log2), in = r - first_s[b];
          chunk = (int)(in / groups);
          t0 = start + ((int)(in - (uint32_t)chunk * groups) << a.tg_log2);
          ntok = min(TG, end - t0);
          // the pages that the loading warp will ask for are on their way to L2
          prefetch_l2(a.block_table + (int64_t)(b0 + b) * a.MB + __umulhi((uint32_t)(chunk * unit_keys), a.page_inv));
        }
        const int taken = __popc(__ballot_sync(0xffffffffu, u < end_units));
        for (int src = 0; src < taken && ok; ++src) {
          const int us = b0 + __shfl_sync(0xffffffffu, b, src), ut0 = __shfl_sync(0xffffffffu, t0, src);
          const int un = __shfl_sync(0xffffffffu, ntok, src), uchunk = __shfl_sync(0xffffffffu, chunk, src);
          const int ustart = __shfl_sync(0xffffffffu, start, src), uend = __shfl_sync(0xffffffffu, end, src);
          const int uL = __shfl_sync(0xffffffffu, L, src);
          const int c0 = uchunk * unit_blocks, uk0 = uchunk * unit_keys;
          const int ulast = min(keys_seen(ut0 + un - 1, ustart, uend, uL, a.causal), uk0 + unit_keys);
          // the blocks behind the sequence's last unit hold no key
          const int blocks = min(unit_blocks, a.C - c0), rest = uk0 + unit_keys >= uL ? a.C - c0 - blocks : 0;
          if (ulast <= uk0) {                             // no token sees these blocks
            for (int i = 0; i < un; ++i)
              for (int c = lane; c < blocks + rest; c += 32) a.out[(int64_t)(ut0 + i) * a.C + c0 + c] = -INFINITY;
            continue;
          }
          ok = finish_unit(ub, uph, nu >= (uint32_t)units);
          if (!ok) break;
          UnitInfo& I = info_s[ub];
          if (lane == 0) {
            I.t0 = ut0;
            I.ntok = un;
            I.k0 = uk0;
            I.last = ulast;
            I.tiles = (ulast - uk0 + kISKeys - 1) / kISKeys;
            I.c0 = c0;
            I.blocks = blocks;
            I.rest = rest;
            I.seq = us;
          }
          if (lane < un) I.seen[lane] = keys_seen(ut0 + lane, ustart, uend, uL, a.causal);
          const uint32_t wbytes = bulk_weights ? (uint32_t)(un * Hp) * 4 : 0u;
          if (wbytes == 0) {
            const float* from = a.w + (int64_t)ut0 * a.H;
#pragma unroll 1
            for (int e = lane; e < un * a.H; e += 32) {
              const int i = quotient(e, a.by_heads);
              gW[ub * q_rows + i * Hp + e - i * a.H] = from[e];
            }
          }
          __syncwarp();
          if (el) {
            mbar_arrive(b_info + 8 * ub);
            // (a group with fewer tokens loads what lies behind them, which no product reads)
            mbar_arrive_expect_tx(b_qfull + 8 * ub, (uint32_t)(q_rows * kDIndex) + wbytes);
            if (wbytes) bulk_load(smem_u32(gW + ub * q_rows), a.w + (int64_t)ut0 * a.H, wbytes, b_qfull + 8 * ub);
            tma_load_3d(sQ + ub * q_rows * kDIndex, &a.tm_q, b_qfull + 8 * ub, 0, 0, ut0);
          }
          __syncwarp();
          ++nu;
          if (++ub == (uint32_t)units) { ub = 0; uph ^= 1; }
        }
        if (taken < 32) {                               // the rest are units of sequences to come
          next += (int64_t)taken * gridDim.x;
          break;
        }
      }
      counted = end_units;
    }
    // the end of the units: the others leave, and the last units' scores are written
    for (int i = 0; i < units && ok; ++i) {
      ok = finish_unit(ub, uph, nu + i >= (uint32_t)units);
      if (i == 0 && ok) {
        if (lane == 0) info_s[ub].ntok = 0;
        __syncwarp();
        if (el) {
          mbar_arrive(b_info + 8 * ub);
          mbar_arrive(b_qfull + 8 * ub);
        }
      }
      if (++ub == (uint32_t)units) { ub = 0; uph ^= 1; }
    }
    if (!ok && lane == 0) {
      // copies in flight land before the CTA leaves: the last fill of each buffer
      volatile uint32_t none = 0u;
      for (uint32_t k = nu > (uint32_t)units ? nu - units : 0; k < nu; ++k)
        mbar_wait(b_qfull + 8 * (k % units), (k / units) & 1, &none, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------------------------------------------------------------------- keys and scales
    const bool el = elect_one();
    const int per = kISKeys / a.box_rows;               // boxes of a tile
    const int per_log2 = __ffs(per) - 1;
    // a lane brings four scales of each tile
    const int my_box = lane * per >> 5, my_row = lane * 4 - my_box * a.box_rows;
    uint32_t ub = 0, uph = 0, slot = 0, ph = 1, filled = 0;
    bool ok = true;
    while (ok) {
      ok = wait(b_info + 8 * ub, uph);
      if (!ok) break;
      const UnitInfo& I = info_s[ub];
      const int ntok = I.ntok, tiles = I.tiles, k0 = I.k0, last = I.last;
      if (ntok == 0) break;
      // the first rows of the unit's boxes, 32 at a time (one to a lane), 32 ahead
      const int32_t* pages = a.block_table + (int64_t)I.seq * a.MB;
      auto row_of = [&](int box) -> int {
        const int tok = k0 + box * a.box_rows;
        if (tok >= last) return -1;
        const int page = (int)__umulhi((uint32_t)tok, a.page_inv), in = tok - page * a.P;
        int pg = __ldg(pages + page);
        if (pg < 0 || pg >= a.num_pages) {
          atomicOr(err, MLA_DEVERR_BLOCK_TABLE);
          pg = 0;
        }
        return pg * a.P + in;
      };
      int rows = row_of(lane), ahead = tiles * per > 32 ? row_of(lane + 32) : -1;
      if (S >= kISTogether) {
        // several tiles at once: a wait, an expected count or a box costs the warp about 100 clocks whether one lane
        // or several make it (a decode step 18.4 us, tile by tile 21.5)
        for (int tile = 0; tile < tiles;) {
          const int at = tile * per & 31;                 // per divides 32
          if (tile > 0 && at == 0) {
            rows = ahead;
            ahead = row_of((tile * per & ~31) + 32 + lane);
          }
          const int some = min(min(kISTogether, tiles - tile), (32 - at) >> per_log2);
          uint32_t my_slot = slot + (uint32_t)lane;       // lanes 0 .. some - 1: a tile each
          const bool wraps = my_slot >= (uint32_t)S;
          if (wraps) my_slot -= S;
          const uint32_t empty = b_kempty + 8 * my_slot, parity = ph ^ (wraps ? 1u : 0u);
          ok = __all_sync(0xffffffffu, lane >= some || mbar_try_wait_sleep(empty, parity, kISFirstWaitNs) ||
                                           wait_longer(empty, parity, smem_u32(&abort_s), err, a.wait_limit_ns));
          if (!ok) break;
          if (lane < some) mbar_arrive_expect_tx(b_kfull + 8 * my_slot, kISSlotBytes);
          const int row = __shfl_sync(0xffffffffu, rows, at + lane);
          uint32_t box_slot = slot + ((uint32_t)lane >> per_log2);
          if (box_slot >= (uint32_t)S) box_slot -= S;
          // a box past the keys starts at the end of the pool and reads zeros
          if (lane < some << per_log2)
            tma_load_2d(sK + box_slot * kISSlotBytes + (lane & (per - 1)) * a.box_rows * kDIndex, &a.tm_k, b_kfull + 8 * box_slot, 0,
                        row >= 0 ? row : a.total_rows);
          for (int k = 0; k < some; ++k) {
            const int srow = __shfl_sync(0xffffffffu, rows, at + (k << per_log2) + my_box);
            if (srow >= 0) copy16(sS + ((filled % kISScales) * kISKeys + lane * 4) * 4, a.scale + srow + my_row);
            arrive_after_copies(b_kfull + 8 * slot);
            ++filled;
            if (++slot == (uint32_t)S) { slot = 0; ph ^= 1; }
          }
          tile += some;
        }
      } else {
        // few slots, as beside large queries: tile by tile (4 tokens of 4 long sequences x 64 heads, four slots, 19.9 us;
        // in the form above, four at once, 23.3; 4 tokens of 64 sequences 18.6 and 22.8)
        for (int tile = 0; tile < tiles; ++tile) {
          const int at = tile * per & 31;                 // per divides 32
          if (tile > 0 && at == 0) {
            rows = ahead;
            ahead = row_of((tile * per & ~31) + 32 + lane);
          }
          const int row = __shfl_sync(0xffffffffu, rows, at + (lane & (per - 1)));
          const int srow = __shfl_sync(0xffffffffu, rows, at + my_box);
          ok = wait(b_kempty + 8 * slot, ph);
          if (!ok) break;
          const uint32_t bar = b_kfull + 8 * slot;
          if (el) mbar_arrive_expect_tx(bar, kISSlotBytes);
          __syncwarp();
          // a box past the keys starts at the end of the pool and reads zeros
          if (lane < per)
            tma_load_2d(sK + slot * kISSlotBytes + lane * a.box_rows * kDIndex, &a.tm_k, bar, 0, row >= 0 ? row : a.total_rows);
          if (srow >= 0) copy16(sS + ((filled % kISScales) * kISKeys + lane * 4) * 4, a.scale + srow + my_row);
          arrive_after_copies(bar);
          ++filled;
          if (++slot == (uint32_t)S) { slot = 0; ph ^= 1; }
        }
      }
      if (++ub == (uint32_t)units) { ub = 0; uph ^= 1; }
    }
    if (!ok && lane == 0) {
      volatile uint32_t none = 0u;
      for (uint32_t f = filled > (uint32_t)S ? filled - S : 0; f < filled; ++f)
        mbar_wait(b_kfull + 8 * (f % S), (f / S) & 1, &none, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp < kISFirst) {
    // ---------------------------------------------------------------------------------- MMAs
    const bool el = elect_one();
    const uint32_t me = (uint32_t)warp - 1;             // the pair of accumulators this warp fills
    const uint32_t acc = tmem + me * 2 * kISColumns, b_full = b_tfull + 8 * me, b_free = b_tempty + 8 * me;
    uint32_t slot = 0, ph = 0, n = 0, mine = 0;         // n: products so far, of both; mine: of this warp
    bool ok = true;
    for (uint32_t qb = 0, qph = 0; ok; qb + 1 == (uint32_t)units ? (qb = 0, qph ^= 1) : ++qb) {
      ok = wait(b_qfull + 8 * qb, qph);
      if (!ok) break;
      // (the same in every lane, which the compiler can use for the descriptors)
      const int ntok = __shfl_sync(0xffffffffu, info_s[qb].ntok, 0), tiles = __shfl_sync(0xffffffffu, info_s[qb].tiles, 0);
      if (ntok == 0) break;
      const uint64_t qd = make_sdesc(sQ + qb * q_rows * kDIndex, 16, 1024, kSwizzle128);
      const bool one = ntok <= sub_tokens;              // one sub-group: a product is two tiles of it
      const int pair = 2 * sub_tokens;
      for (int tile = 0; tile < tiles && ok; tile += one ? 2 : 1) {
        const bool two = one && tile + 1 < tiles;
        const uint32_t slot1 = slot + 1 == (uint32_t)S ? 0 : slot + 1, ph1 = slot1 == 0 ? ph ^ 1 : ph;
        ok = wait(b_kfull + 8 * slot, ph) && (!two || wait(b_kfull + 8 * slot1, ph1));
        if (!ok) break;
        const uint64_t kd = make_sdesc(sK + slot * kISSlotBytes, 16, 1024, kSwizzle128);
        for (int t = 0; t < ntok; t += pair, ++n) {
          if ((n & 1) != me) continue;
          ok = wait(b_free, (mine & 1) ^ 1);
          if (!ok) break;
          ++mine;
          tc_fence_after();
          if (el) {
            const uint32_t idesc = make_idesc(128, (uint32_t)(min(pair, ntok - t) * Hp), 0, 0, 0);
            const uint64_t qt = qd + (uint64_t)((uint32_t)(t * Hp * kDIndex) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_f8(acc, kd + 2 * k, qt + 2 * k, idesc, k > 0);
            if (two) {
              const uint64_t kd1 = make_sdesc(sK + slot1 * kISSlotBytes, 16, 1024, kSwizzle128);
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_f8(acc + kISColumns, kd1 + 2 * k, qt + 2 * k, idesc, k > 0);
            }
            umma_commit(b_full);
            mbar_arrive(b_full);
          }
          __syncwarp();
        }
        if (!ok) break;
        // both issuing warps see every tile land before they give its slot back
        if (el) {
          umma_commit(b_kempty + 8 * slot);
          if (two) umma_commit(b_kempty + 8 * slot1);
          if (tile + (one ? 2 : 1) >= tiles) umma_commit(b_qempty + 8 * qb);
        }
        __syncwarp();
        if (two) { slot = slot1; ph = ph1; }
        if (++slot == (uint32_t)S) { slot = 0; ph ^= 1; }
      }
    }
    if (!ok) {
      // the MMAs issued so far complete before tensor memory is freed
      volatile uint32_t none = 0u;
      if (el) umma_commit(b_drain + 8 * me);
      if (lane == 0) mbar_wait(b_drain + 8 * me, 0, &none, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- sums over heads, maxima over keys
    const uint32_t wg = (uint32_t)(warp - kISFirst) >> 2, set = wg >> 1, half = wg & 1;   // pair, and which of it
    const int quad = warp & 3;                          // tensor-memory lanes 32 quad ..
    const int et = threadIdx.x - 32 * kISFirst;
    const uint32_t acc_set = tmem + ((uint32_t)(quad * 32) << 16) + set * 2 * kISColumns;
    const uint32_t b_full = b_tfull + 8 * set, b_free = b_tempty + 8 * set;
    // errors that only the device can see
    for (int b = blockIdx.x * (32 * kISWarps) + et; b < a.B; b += gridDim.x * (32 * kISWarps)) {
      const uint32_t bad = ragged_errors(a.cu_q, a.seq_lens, b, a.T, a.max_len);
      if (bad) atomicOr(err, bad);
    }
    uint32_t nt = 0, n = 0, taken = 0;                  // tiles and products so far, products of this pair
    bool ok = !(a.test_stall && !wait(b_never, 0));
    for (uint32_t qb = 0, qph = 0; ok; qb + 1 == (uint32_t)units ? (qb = 0, qph ^= 1) : ++qb) {
      ok = wait(b_qfull + 8 * qb, qph);
      if (!ok) break;
      const UnitInfo& I = info_s[qb];
      const int ntok = I.ntok, tiles = I.tiles;
      if (ntok == 0) break;
      int* mine = best + qb * maxima;
      const bool one = ntok <= sub_tokens;
      const int turns = ntok > 2 * sub_tokens ? 2 : 1;  // products of a tile
      const int products = one ? (tiles + 1) >> 1 : tiles * turns;
      for (int m = (int)((n + set) & 1); m < products; m += 2, ++taken) {
        const int tile = one ? 2 * m + (int)half : m >> (turns - 1);
        const int t0 = one ? 0 : (2 * (m & (turns - 1)) + (int)half) * sub_tokens;
        ok = wait(b_full, taken & 1);
        if (!ok) break;
        // the accumulator has been read
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_free);
        };
        if (tile >= tiles || t0 >= ntok) {              // the pair's second half is empty
          release();
          continue;
        }
        const uint32_t gt = nt + (uint32_t)tile;
        const uint32_t acc = acc_set + half * (uint32_t)(one ? kISColumns : sub_tokens * Hp);
        tc_fence_after();
        const float ks = gS[(gt % kISScales) * kISKeys + quad * 32 + lane];
        const int in = tile * kISKeys + quad * 32 + lane;     // key within the unit
        const int key = I.k0 + in;
        const int toks = min(sub_tokens, ntok - t0);
        const float* w = gW + qb * q_rows + t0 * Hp;
        int* to = mine + t0 * a.unit_blocks + (int)__umulhi((uint32_t)(kWhole ? in - lane : in), a.block_inv);
        float keep = -INFINITY;
        uint64_t s[4];
        // (the warps of a scheduler cover each other's loads: a second buffer changes nothing)
        auto finish = [&](int i, auto masked) {         // token i's score of this key, and its maximum over keys
          float x = sum8(s) * ks;
          if (decltype(masked)::value && key >= I.seen[t0 + i]) x = -INFINITY;
          if (kWhole) {
            x = warp_max(x);
            if (lane == i) keep = x;
          } else {
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if ((lane & 7) == 0 && x > -INFINITY) atomicMax(to + i * a.unit_blocks, ordered(x));
          }
        };
        auto tokens = [&](int i, auto masked) {         // kAtOnce of them
          float v[32];
#pragma unroll
          for (int c = 0; c < PT; ++c) {
            const int at = (i * PT + c) * CS;
            tmem_ld32(acc + at, v);
            tmem_wait_ld();
            if (c + 1 == PT && i + kAtOnce >= toks) release();
            if (c == 0) add_heads<CS, true>(v, w + at, s);
            else add_heads<CS, false>(v, w + at, s);
          }
          finish(i, masked);
          if (kAtOnce == 2 && (!decltype(masked)::value || i + 1 < toks)) {
            add_heads<CS, true>(v + 32 - CS, w + (i + 1) * CS, s);
            finish(i + 1, masked);
          }
        };
        // a full accumulator whose tokens see all keys of the tile, the usual case, has code of its own
        if (toks == kFull && I.k0 + (tile + 1) * kISKeys <= I.seen[t0]) {
#pragma unroll
          for (int i = 0; i < kFull; i += kAtOnce) tokens(i, std::false_type{});
        } else {
          for (int i = 0; i < toks; i += kAtOnce) tokens(i, std::true_type{});
        }
        if (kWhole && lane < toks && keep > -INFINITY) atomicMax(to + lane * a.unit_blocks, ordered(keep));
      }
      if (!ok) break;
      n += (uint32_t)products;
      nt += (uint32_t)tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_qempty + 8 * qb);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kISTmem);
}

cudaError_t index_scores_prepare() {
  for (auto* kernel : {index_scores_kernel<16, 1, false>, index_scores_kernel<32, 1, false>, index_scores_kernel<32, 2, false>,
                       index_scores_kernel<32, 4, false>, index_scores_kernel<16, 1, true>, index_scores_kernel<32, 1, true>,
                       index_scores_kernel<32, 2, true>, index_scores_kernel<32, 4, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kISSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Columns of a token, and tokens of a group: as many as sequences have on average (a power of two), up to four
// sub-groups. One size for all units keeps their queries in one box. Where sequences are alike that is the right one;
// in a batch of both kinds, 64 heads, us, together / a call for each: 127 single tokens and a prompt of 2048 tokens
// over 24 K keys 413 / 21 + 404, over none 48 / 21 + 29; 255 and a prompt of 512 over 8 K (groups of two, which fetch
// the prompt's keys four times as often) 99 / 40 + 44, over 24 K 208 / 40 + 105.
void index_scores_group(int T, int B, int H, int* columns, int* tokens) {
  *columns = 16;
  while (*columns < H) *columns *= 2;
  const int most_tokens = 2 * kISIssuers * (kISColumns / *columns);
  *tokens = 1;
  while (*tokens < T / B && *tokens < most_tokens) *tokens *= 2;
}

cudaError_t launch_index_scores(IndexScoreArgs a, int num_sms, cudaStream_t s) {
  int Hp;
  index_scores_group(a.T, a.B, a.H, &Hp, &a.TG);
  const int sub_tokens = kISColumns / Hp;
  a.tg_log2 = 0;
  while (1 << a.tg_log2 < a.TG) ++a.tg_log2;
  const bool many = a.TG > sub_tokens;
  a.q_rows = a.TG * Hp;
  // A unit: about 24 to a CTA (6 of a decode step), of 512 to 8192 keys (1024), as far as they are whole blocks and
  // whole tiles (blocks of 1016 keys: 16256) and their maxima fit (256 keys for 32 tokens and blocks of 8).
  int lcm = a.block;
  while (lcm % kISKeys != 0) lcm += a.block;
  const int64_t groups = (a.T + a.TG - 1) / a.TG;
  const int64_t top = many ? 8192 : 1024;
  int64_t keys = groups * a.max_len / ((many ? 24 : 6) * (int64_t)num_sms);
  keys = keys < 512 ? 512 : keys > top ? top : keys;
  int64_t m = keys / lcm;
  const int64_t most = kISBest / ((int64_t)a.TG * (lcm / a.block));
  m = m > most ? most : m;
  if (m < 1) m = 1;
  // Where the contexts may come to no more than 32 tiles a CTA, the kernel takes the size that suits their actual
  // lengths, from one step (128 keys where blocks divide a tile) up to 1024 keys: 4 tokens of 4 sequences of 33-131 K
  // 18.9 us instead of 22.5, 1 to 4 sequences of 4 K 6.2 instead of 7.2; 0.5 us on the GPU, which a step of 121
  // sequences would not get back
  a.choose = a.B <= kISSeqs && groups * a.max_len <= (int64_t)32 * kISKeys * num_sms ? 1 : 0;
  int64_t cap = a.choose ? (1024 / lcm < most ? 1024 / lcm : most) : m;
  cap = cap < m ? m : cap;
  a.step_blocks = lcm / a.block;
  a.step_tiles = lcm / kISKeys;
  a.usual_blocks = (int)m * a.step_blocks;
  a.unit_blocks = (int)cap * a.step_blocks;
  a.block_inv = (uint32_t)((((uint64_t)1 << 32) + a.block - 1) / a.block);   // keys of a unit x block < 2^32
  a.by_blocks = 0xFFFFFFFFu / (uint32_t)a.unit_blocks;
  a.by_heads = 0xFFFFFFFFu / (uint32_t)a.H;
  a.page_inv = (uint32_t)((((uint64_t)1 << 32) + a.P - 1) / a.P);            // a key of a sequence x P < 2^32
  // (queries of 256 rows: two buffers leave eight slots for keys instead of four, and 4 tokens of 4 long sequences x 64
  // heads take 22.2 us instead of 19.9, of 64 sequences 21.4 instead of 18.6: short units want their queries early)
  a.units = a.q_rows <= kISManyRows ? kISMaxUnits : 2;
  const int fixed = is_fixed_bytes(a.units, a.q_rows, a.TG * a.unit_blocks);
  a.key_slots = is_key_slots(a.units, a.q_rows, a.TG * a.unit_blocks);
  if (a.key_slots > kISMaxSlots) a.key_slots = kISMaxSlots;
  const int smem = fixed + a.key_slots * kISSlotBytes;
  const int64_t total = ((int64_t)a.T / a.TG + a.B) * ((a.C + a.step_blocks - 1) / a.step_blocks);   // units at most
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(total < num_sms ? total : num_sms));
  a.by_grid = 1.f / (float)cfg.gridDim.x;
  cfg.blockDim = dim3(kISThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    return Hp == 16   ? cudaLaunchKernelEx(&cfg, index_scores_kernel<16, 1, kWhole>, a)
           : Hp == 32 ? cudaLaunchKernelEx(&cfg, index_scores_kernel<32, 1, kWhole>, a)
           : Hp == 64 ? cudaLaunchKernelEx(&cfg, index_scores_kernel<32, 2, kWhole>, a)
                      : cudaLaunchKernelEx(&cfg, index_scores_kernel<32, 4, kWhole>, a);
  };
  return a.block % 32 == 0 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace mla
