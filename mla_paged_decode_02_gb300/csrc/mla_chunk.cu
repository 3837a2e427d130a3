// mla_chunk.cu — attention of a ragged batch of new tokens over the paged latent cache, on CTA
// pairs (sm_103a: a cluster of two CTAs on two SMs, tcgen05 MMAs with cta_group::2).
//
// For a block of 128 query rows of one sequence (row = token * H + head; the token sees the
// first n_r keys) the kernel computes  s = scale q.K,  p = exp(s - m),  O = sum p V,  l = sum p
// in one pass over the keys, with a running reference m (moved up only when a score exceeds it by
// more than a factor of 2^8, E4M3 2^4; O is rescaled then), and leaves out = O / l, lse = m + ln l.
//
// Rows on M. The float32 accumulator of 128 rows x 512 columns fills one SM's tensor memory, so
// a pair shares it: CTA k holds rows 64 k .. 64 k + 63 (M = 128 over the pair), and every MMA
// has N = 256, half of its B operand from each CTA. Both are full rate on this GPU: 37 ns per
// K = 16 step, like M = 256 with N = 128 (N = 128 here would cost 26 ns, more than half).
//   QK^T  N = 256 keys of a tile: CTA k holds keys 128 k .. as B;
//   PV    N = 256 value columns, twice (j = 0, 1): CTA k holds columns 256 k + 128 j .. as B.
// An SM's accumulator rows then hold, in tensor-memory lane l, row l % 64: N columns 0..127 in
// lanes 0..63 and 128..255 in lanes 64..127. So a thread owns a quarter of the keys of one row, the
// softmax stays inside the CTA (four threads compare maxima), and P needs no exchange.
// Tensor memory per CTA: S 2 x 128 columns, O 2 x 128.
//
// Shared memory per CTA: 64 query rows (72 KB), P (64 rows x 256 keys, 32 KB), and seven 16 KB slots
// in two rings: keys (128 keys x 128 bytes of the row) and values (this CTA's 256 columns of 32 or,
// E4M3, 64 keys). The 512-byte value pieces come from L2: the peer has just read those keys.
//
// Two issuing warps, each with a ring and a producer, so that QK^T of tile n + 1 (of the next unit
// too) overlaps the softmax and PV of tile n. They stay converged, every lane waiting and one
// elected lane issuing: with a wait before every four MMAs an issuing thread in a branch of its
// own takes 56 ns per MMA, an elected lane of a converged warp 36 (the rate of the tensor core).
//
// The FP8 cache. As in the decode kernels, the MMAs read the E4M3 bytes as they land
// (kind::f8f6f4) against q and P written as two terms each (hi + lo). q, scaled per row by a power of
// two, is two E4M3 terms: exact down to 2^-10 of the row's largest value, off by at most 2^-17 of
// it below. P times 2^4 is an E4M3 and an E5M2 term: 8 significant bits for weights down to 2^-10 of
// the reference; smaller ones are off by at most 2^-18 of it and by 1/8 of themselves, and end at
// 2^-21. The normaliser sums the unrounded weights, so what P loses the result loses: with a
// reference that only rises, one strong early key over a long even context would leave most of the
// weight in terms of few bits. So every 4 tiles the reference also moves down, to the largest
// score of those 1024 keys, when that lies more than 2^4 below it; O and l grow instead (float32
// holds the 2^60 that the reference may fall in all). Few keys' weights are then of few bits, however
// many there are: with strong keys 6 to 13 natural-log units above 32 K and 128 K others the 2-norm of
// the error is 0.002 to 0.004 of the result (0.05 to 0.86 with two E4M3 terms and a reference that only
// rises). 128-token pieces x 128 heads over 32 K keys take 1482 us so and 1465 without; looking every 8
// tiles, 1480 us and errors up to 0.007.
//
// Masks. Scores of keys a row does not see are selected away by index, whatever they hold. In
// the PV product such keys meet P = 0, and 0 x NaN is NaN: value slots with a key that some row
// of the block does not see are put right when they land: zeros over rows no row sees and over
// non-finite values of rows that only some see (a row that does see such a key has a
// non-finite score there, which makes its result NaN without the value; a score of -inf gives
// the key weight 0). Boxes past the last key start at the end of the pool, so TMA fills zeros.
//
// Roles (512 threads): warp 0 loads q and keys, warp 2 values; warps 1 and 3 of the even CTA issue
// QK^T and PV; warps 4-11 softmax, four threads to a row; warps 12-15 (E4M3) the split of q, and the
// epilogue. Every wait is bounded; a stall sets the device error word, and both CTAs drain and
// leave through a cluster barrier.
//
// Ordering between the CTAs. What a thread of the odd CTA writes for the MMAs (P, value slots put
// right, the terms of q) it releases at cluster scope, and the issuing warps acquire at that scope.
// Signals that a tensor-memory buffer was read are relaxed: they publish no memory, and the reads
// have completed (tcgen05.wait::ld) before them.
//
// Bound by the tensor cores: 512 tokens x 128 heads over 8 K keys, bf16, 627 us cold (1920 TFLOP/s,
// tensor cycles 88% busy) and 0.70-0.73 ms one after another under the power limit; 128-token
// pieces x 128 heads over 32 K keys, E4M3, 1316 us cold (93%). Short causal blocks are bound by what a
// block adds at its ends: 8 prompts of 150 to 2000 tokens x 16 heads, 14 blocks per pair, 169 us (58%).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "mla_chunk.h"
#include "mla_ptx.cuh"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kCSlots = 7;                       // key and value slots
constexpr int kCSlot = 16384;
constexpr int kCQChunk = 8192;                   // 64 rows x 64 columns bf16
constexpr int kCQBytes = 9 * kCQChunk;
constexpr int kCPBytes = 64 * kChunkTile * 2;    // bf16, or E4M3 hi and lo
constexpr int kCThreads = 512;
constexpr int kCTmemCols = 512;
constexpr int kCOCol = 256;                      // O at columns 256 + 128 j
constexpr int kCDynBytes = 1024 + kCQBytes + kCPBytes + kCSlots * kCSlot;
constexpr int kCSmemLimit = 232448;
constexpr int kCStaticBudget = 6144;
static_assert(kCDynBytes + kCStaticBudget <= kCSmemLimit, "shared memory budget");
constexpr float kCLog2e = 1.4426950408889634f;
constexpr float kCLn2 = 0.6931471805599453f;

template <bool FP8>
struct ChunkCfg {
  static constexpr int kKeySlots = FP8 ? 5 : 9;          // 128 bytes of the key row each
  static constexpr int kSlotKeys = FP8 ? 64 : 32;        // keys of a value slot
  static constexpr int kValueChunks = FP8 ? 2 : 4;       // 128-byte pieces of its rows
  // a tile takes 9 key and 8 value slots (bf16) or 5 and 4; the better split of the seven, measured
  // against 4 + 3 and 3 + 4: bf16 prompts 188 -> 181 us; E4M3 mixed step 98 against 103 us, prompts
  // 206 to 217 against 240, single tokens alone 63 against 66, 32 K keys x 128 heads 1453 against 1474
  static constexpr int kKRing = FP8 ? 4 : 3, kVRing = kCSlots - kKRing;
  static constexpr float kRescaleLog2 = FP8 ? 4.f : 8.f;
  static constexpr float kPOffLog2 = FP8 ? 4.f : 0.f;
  // E4M3: every kWindow tiles the reference also moves down to the largest score of those tiles,
  // if that is more than kLowerLog2 below it, but to no more than kSpanLog2 below its highest value.
  static constexpr int kWindow = 4;
  static constexpr float kLowerLog2 = 4.f, kSpanLog2 = 60.f;
  static_assert(kSlotKeys * kValueChunks * 128 == kCSlot, "value slot");
};

struct CUnit {
  int b, row0, srow0, tb, te, slot, len, vis, nrows;
  int lo, hi;    // keys every row sees; keys some row sees
};

__device__ __forceinline__ CUnit load_cunit(const ChunkArgs& a, int u) {
  const int4* p = reinterpret_cast<const int4*>(a.units + u);
  const int4 x = p[0], y = p[1];
  CUnit r;
  r.b = x.x;
  r.row0 = x.y;
  r.srow0 = x.z;
  r.tb = x.w & 0xFFFF;
  r.te = (int)((unsigned)x.w >> 16);
  r.slot = y.x;
  r.len = y.y;
  r.vis = y.z;
  r.nrows = y.w;
  if (a.causal) {
    r.lo = max(0, r.vis + r.srow0 / a.H);
    r.hi = max(0, r.vis + (r.srow0 + r.nrows - 1) / a.H);
  } else {
    r.lo = r.hi = r.len;
  }
  return r;
}

// value slots of tile `tile` of a block that sees hi keys
template <int kSlotKeys>
__device__ __forceinline__ int value_slots(int hi, int tile) {
  const int left = hi - tile * kChunkTile;
  return left >= kChunkTile ? kChunkTile / kSlotKeys : (left + kSlotKeys - 1) / kSlotKeys;
}

// First cache row of the 8 keys 8 lane .. of a tile, for the boxes that start there: past the keys
// the block sees the pool's end (TMA fills such a box with zeros); a block-table entry outside the
// pool reads page 0 (the combine kernel reports it).
__device__ __forceinline__ int tile_row(const ChunkArgs& a, const CUnit& U, int tile, int lane) {
  const int tok = tile * kChunkTile + 8 * lane;
  if (tok >= U.hi) return a.total_rows;
  const int page = tok / a.P, in = tok - page * a.P;
  const int pg = __ldg(a.block_table + (int64_t)U.b * a.MB + page);
  return (pg < 0 || pg >= a.num_pages) ? in : pg * a.P + in;
}

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar_cluster, int32_t c0,
                                                 int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(c0), "r"(c1) : "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// zero over the non-finite values of 4 bytes
template <bool FP8>
__device__ __forceinline__ uint32_t finite_word(uint32_t w) {
  if (FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((w >> (8 * i)) & 0x7Fu) == 0x7Fu) w &= ~(0xFFu << (8 * i));
  } else {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  }
  return w;
}

// 32 bytes of a thread: one store where `wide` (the address is a multiple of 32), else two of 16
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  } else {
    uint4* q = reinterpret_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The rest of a wait that acquires at cluster scope (as wait_longer): for the issuing warps, whose MMAs
// read what threads of both CTAs wrote.
__device__ __noinline__ bool wait_longer_cluster(uint32_t bar, uint32_t parity, uint32_t abort_s, uint32_t peer,
                                                 uint32_t* err, uint64_t limit_ns) {
  volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(__cvta_shared_to_generic(abort_s));
  const bool ok = mbar_wait_cluster(bar, parity, flag, err, MLA_DEVERR_TIMEOUT, limit_ns);
  if (!ok) st_cluster_u32(map_to_rank(abort_s, peer), 1u);
  return ok;
}

// The rest of a wait that was not over at the first look, out of line: some thirty waits share the
// instruction cache. A wait that fails also raises the peer's abort flag, so that its waits end.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, uint32_t abort_s, uint32_t peer, uint32_t* err,
                                         uint64_t limit_ns) {
  volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(__cvta_shared_to_generic(abort_s));
  const bool ok = mbar_wait(bar, parity, flag, err, MLA_DEVERR_TIMEOUT, limit_ns);
  if (!ok) st_cluster_u32(map_to_rank(abort_s, peer), 1u);
  return ok;
}

// 64 bytes (16 words) of the rows of two neighbouring lanes: they swap halves, so that a pair
// writes 64 contiguous bytes of the even lane's row and then of the odd lane's. `p` points to the
// even lane's row, plus 32 bytes in the odd lane; keep0, keep1: whether those rows are stored.
// (With each lane writing 16 bytes of its own row at a time, the first tile of the next unit ran about
// 3 us late, and 8 prompts of 16 heads took 234 us, so 222; the likely reason is the load/store
// path, which the barriers of all roles share.)
__device__ __forceinline__ void store_pair64(uint8_t* p, size_t row_bytes, uint32_t* w, bool odd, bool keep0, bool keep1,
                                             bool wide) {
#pragma unroll
  for (int y = 0; y < 8; ++y) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[y] : w[8 + y], 1);
    if (odd) w[y] = got;
    else w[8 + y] = got;
  }
  if (keep0) store32(p, w, wide);
  if (keep1) store32(p + row_bytes, w + 8, wide);
}

// whether all values of 16 bytes are finite: no exponent (bf16) or magnitude (E4M3) is all ones
template <bool FP8>
__device__ __forceinline__ bool finite_words(const uint4& v) {
  // adding one to an all-ones field carries into the bit above it, which the mask has cleared
  constexpr uint32_t kMask = FP8 ? 0x7F7F7F7Fu : 0x7F807F80u, kOne = FP8 ? 0x01010101u : 0x00800080u;
  constexpr uint32_t kCarry = FP8 ? 0x80808080u : 0x80008000u;
  const uint32_t c = (((v.x & kMask) + kOne) | ((v.y & kMask) + kOne)) | (((v.z & kMask) + kOne) | ((v.w & kMask) + kOne));
  return (c & kCarry) == 0u;
}

// One lane of a converged warp. The issuing warps stay converged around it, their barrier waits
// and descriptor arithmetic warp-uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ float max64(const float* s) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < 64; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = i + 4 + j < 64 ? fmaxf(m[j], fmaxf(s[i + j], s[i + 4 + j])) : fmaxf(m[j], s[i + j]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// (x, y) * c + d and pairwise sums, two values per instruction
__device__ __forceinline__ void fma2(float& x, float& y, float c, float d) {
  asm("{\n\t.reg .b64 v, w, z;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 v, v, w, z;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y) : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ float sum32(const float* s) {
  float a[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < 32; i += 4) {
    add2(a[0], a[1], s[i], s[i + 1]);
    add2(a[2], a[3], s[i + 2], s[i + 3]);
  }
  return (a[0] + a[1]) + (a[2] + a[3]);
}

// 32 lanes x 32 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
}

}  // namespace

template <bool FP8, bool kSub>
__global__ void __launch_bounds__(kCThreads, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  using Cfg = ChunkCfg<FP8>;
  constexpr int KS = Cfg::kKeySlots, VK = Cfg::kSlotKeys, VC = Cfg::kValueChunks;
  constexpr int kKRing = Cfg::kKRing, kVRing = Cfg::kVRing;
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ __align__(8) uint64_t bar_kfull[kKRing], bar_kempty[kKRing], bar_vfull[kVRing], bar_vempty[kVRing], bar_aux[kVRing];
  __shared__ __align__(8) uint64_t bar_qfull, bar_qempty, bar_qraw, bar_qsc, bar_qfree;
  __shared__ __align__(8) uint64_t bar_sfull[2], bar_sempty[2], bar_p[2], bar_pv[2], bar_oempty, bar_stat, bar_statfree, bar_drain, bar_never;
  __shared__ uint32_t tmem_base_s, abort_s;
  __shared__ float qf_s[64];                 // E4M3: 2^-e of this CTA's rows
  __shared__ float mx_s[2][256], sum_s[256], ref_s[128];
  __shared__ float top_s[FP8 ? 256 : 1];     // E4M3: a thread's highest reference of the unit

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;

  const uint32_t raw = smem_u32(dsmem_raw);
  const uint32_t sQ = (raw + 1023u) & ~1023u;
  uint8_t* gQ = dsmem_raw + (sQ - raw);
  const uint32_t sP = sQ + kCQBytes, sK = sP + kCPBytes, sV = sK + kKRing * kCSlot;
  uint8_t* gP = gQ + kCQBytes;
  uint8_t* gV = gP + kCPBytes + kKRing * kCSlot;

  const uint32_t b_kfull = smem_u32(bar_kfull), b_kempty = smem_u32(bar_kempty);
  const uint32_t b_vfull = smem_u32(bar_vfull), b_vempty = smem_u32(bar_vempty), b_aux = smem_u32(bar_aux);
  const uint32_t b_sempty = smem_u32(bar_sempty);
  const uint32_t b_qfull = smem_u32(&bar_qfull), b_qempty = smem_u32(&bar_qempty), b_qraw = smem_u32(&bar_qraw);
  const uint32_t b_qsc = smem_u32(&bar_qsc), b_qfree = smem_u32(&bar_qfree);
  const uint32_t b_sfull = smem_u32(bar_sfull), b_p = smem_u32(bar_p), b_pv = smem_u32(bar_pv);
  const uint32_t b_oempty = smem_u32(&bar_oempty), b_stat = smem_u32(&bar_stat), b_statfree = smem_u32(&bar_statfree);
  const uint32_t b_drain = smem_u32(&bar_drain), b_never = smem_u32(&bar_never);
  volatile uint32_t* abort_flag = &abort_s;
  uint32_t* err = a.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKRing; ++i) {
      mbar_init(b_kfull + 8 * i, 1);      // the even CTA's producer, with both CTAs' bytes
      mbar_init(b_kempty + 8 * i, 1);     // the issuer's commit (both CTAs)
    }
    for (int i = 0; i < kVRing; ++i) {
      mbar_init(b_vfull + 8 * i, 1);
      mbar_init(b_vempty + 8 * i, 1);
      mbar_init(b_aux + 8 * i, 1);        // a slot that is fixed before it counts as full
    }
    mbar_init(b_qfull, FP8 ? 2 : 1);      // bf16: as b_kfull; E4M3: the converters of both CTAs
    mbar_init(b_qempty, 1);
    mbar_init(b_qraw, 1);
    mbar_init(b_qsc, 1);
    mbar_init(b_qfree, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_sempty + 8 * i, 16);     // both CTAs' softmax warps
      mbar_init(b_p + 8 * i, 2);          // half i of P's keys: both CTAs' softmax
      mbar_init(b_pv + 8 * i, 1);
    }
    mbar_init(b_oempty, 2);               // both CTAs' epilogue
    mbar_init(b_stat, 256);
    mbar_init(b_statfree, 128);
    mbar_init(b_drain, 2);                // both issuers
    mbar_init(b_never, 1);
    abort_s = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (warp == 0) tmem_alloc_pair(smem_u32(&tmem_base_s), kCTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                         // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  griddep_wait();

  const int u0 = a.cta_first[pair], u1 = a.cta_first[pair + 1];
  auto lead = [&](uint32_t addr) { return map_to_rank(addr, 0); };
  // a failed wait also raises the peer's abort flag, so that its waits end too
  auto fail_peer = [&]() { st_cluster_u32(map_to_rank(smem_u32(&abort_s), peer), 1u); };
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    const bool ok = mbar_wait(bar, parity, abort_flag, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
    if (!ok) fail_peer();
    return ok;
  };

  // the same by every lane of a warp that stays converged
  auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) ||
                                       wait_longer(bar, parity, smem_u32(&abort_s), peer, err, a.wait_limit_ns));
  };

  // the same for what the other CTA's threads wrote
  auto wait_issue = [&](uint32_t bar, uint32_t parity) -> bool {
    const bool ok = __all_sync(0xffffffffu, mbar_look_cluster(bar, parity) ||
                                                wait_longer_cluster(bar, parity, smem_u32(&abort_s), peer, err, a.wait_limit_ns));
    fence_acquire_shared();
    return ok;
  };

  // The launch gives every thread 128 registers. The epilogue's threads hold 256 columns of a row
  // as bf16: 72 + 2 x 112 + 216 = 4 x 128.
  if (warp < 4) {
    regs_lower<72>();
    if (warp == 0) {
      // ================================================================== q and keys
      // one thread issues two boxes per slot; pages smaller than 64 rows: lane i issues box i.
      // Every slot takes the same bytes from both CTAs.
      const int kbox = kSub ? a.k_box : 64;
      const int nk = 128 / kbox;                          // boxes of a key slot
      const bool el = elect_one();
      uint32_t slot = 0, ph = 1, uq = 0;
      bool ok = true;
      auto load = [&](uint32_t dst, uint32_t bar, int row, int c) {
        if (FP8) tma_load_2d_pair(dst, &a.tm_k, bar, 128 * c, row);
        else tma_load_3d_pair(dst, &a.tm_k, bar, 0, row, c);
      };
      const uint32_t lb = lead(b_kfull);
      for (int u = u0; u < u1 && ok; ++u) {
        const CUnit U = load_cunit(a, u);
        if (U.te == U.tb) continue;
        int rows = tile_row(a, U, U.tb, lane);
        ok = wait_warp(b_qempty, (uq & 1) ^ 1);
        if (!ok) break;
        if (el) {
          const int32_t q0 = U.row0 + 64 * (int)rank;
          if (FP8) {
            mbar_arrive_expect_tx(b_qraw, kCQBytes);
            tma_load_3d(sQ, &a.tm_q, b_qraw, 0, q0, 0);
          } else {
            if (leader) mbar_arrive_expect_tx(b_qfull, 2 * kCQBytes);
            tma_load_3d_pair(sQ, &a.tm_q, lead(b_qfull), 0, q0, 0);
          }
        }
        ++uq;
        for (int tile = U.tb; tile < U.te; ++tile) {
          // the next tile's page numbers are on their way while this tile's keys are issued
          const int next_rows = tile + 1 < U.te ? tile_row(a, U, tile + 1, lane) : 0;
          const int r0 = __shfl_sync(0xffffffffu, rows, 16 * (int)rank), r1 = __shfl_sync(0xffffffffu, rows, 16 * (int)rank + 8);
          const int row = __shfl_sync(0xffffffffu, rows, 16 * (int)rank + (lane < nk ? lane * (kbox >> 3) : 0));
#pragma unroll 1
          for (int c = 0; c < KS; ++c) {
            ok = wait_warp(b_kempty + 8 * slot, ph);
            if (!ok) break;
            const uint32_t dst = sK + slot * kCSlot, bar = lb + 8 * slot;
            if (el) {
              if (leader) mbar_arrive_expect_tx(b_kfull + 8 * slot, 2 * kCSlot);
              if (!kSub) {
                load(dst, bar, r0, c);
                load(dst + kCSlot / 2, bar, r1, c);
              }
            }
            if (kSub && lane < nk) load(dst + (uint32_t)(lane * kbox) * 128u, bar, row, c);
            if (++slot == kKRing) {
              slot = 0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          rows = next_rows;
        }
      }
      // after an abort the odd CTA cannot observe its own loads (they count on the even CTA's
      // barriers): the producers wait 50 us, far longer than a load takes, before leaving
      if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
      }
    } else if (warp == 2) {
      // ================================================================== values
      const int vbox = kSub ? a.v_box : VK;
      const int nvr = VK / vbox;                          // boxes down a value slot
      const int nv = nvr * VC;
      const bool el = elect_one();
      uint32_t slot = 0, ph = 1;
      bool ok = true;
      const uint32_t lb = lead(b_vfull);
      // a slot with a key that some row does not see (in the last one or two tiles of a block) is
      // loaded on a barrier of this CTA, put right when it has landed, and then counted as full
      uint32_t aux_phase = 0;                             // a bit per slot
      auto load = [&](uint32_t dst, bool fix, int row, int col) {   // col: 128-byte piece of the row
        if (fix) {
          if (FP8) tma_load_2d(dst, &a.tm_v, b_aux + 8 * slot, 128 * col, row);
          else tma_load_3d(dst, &a.tm_v, b_aux + 8 * slot, 0, row, col);
        } else {
          if (FP8) tma_load_2d_pair(dst, &a.tm_v, lb + 8 * slot, 128 * col, row);
          else tma_load_3d_pair(dst, &a.tm_v, lb + 8 * slot, 0, row, col);
        }
      };
      const int c0 = VC * (int)rank;
      for (int u = u0; u < u1 && ok; ++u) {
        const CUnit U = load_cunit(a, u);
        if (U.te == U.tb) continue;
        int rows = tile_row(a, U, U.tb, lane);
        for (int tile = U.tb; tile < U.te; ++tile) {
          const int next_rows = tile + 1 < U.te ? tile_row(a, U, tile + 1, lane) : 0;
          const int n = value_slots<VK>(U.hi, tile);
          int key = tile * kChunkTile;
          const int i = lane % nvr, c = lane / nvr;       // kSub: this lane's box i of piece c
#pragma unroll 1
          for (int s = 0; s < n; ++s) {
            const int r0 = __shfl_sync(0xffffffffu, rows, s * VK >> 3);
            const int row = kSub ? __shfl_sync(0xffffffffu, rows, (s * VK + (lane < nv ? i * vbox : 0)) >> 3) : 0;
            key += VK;
            const bool fix = key > U.lo;
            ok = wait_warp(b_vempty + 8 * slot, ph);
            if (!ok) break;
            const uint32_t dst = sV + slot * kCSlot;
            if (el) {
              if (leader) mbar_arrive_expect_tx(b_vfull + 8 * slot, 2 * kCSlot);
              if (fix) mbar_arrive_expect_tx(b_aux + 8 * slot, kCSlot);
              if (!kSub) {
                load(dst, fix, r0, c0);                            // bf16: four pieces in one box
                if (FP8) load(dst + kCSlot / 2, fix, r0, c0 + 1);
              }
            }
            if (kSub) {
              __syncwarp();
              if (lane < nv) load(dst + (uint32_t)(c * VK + i * vbox) * 128u, fix, row, c0 + c);
            }
            if (fix) {
              const int first_key = key - VK;
              ok = wait_warp(b_aux + 8 * slot, (aux_phase >> slot) & 1);
              if (!ok) break;
              aux_phase ^= 1u << slot;
              uint8_t* g = gV + slot * kCSlot;
              // rows [lo, hi) of the slot keep their finite values, rows from hi on become zeros
              const int lo = max(0, U.lo - first_key), hi = min(VK, U.hi - first_key);
              for (int idx = lane; idx < (hi - lo) * 8; idx += 32) {
#pragma unroll
                for (int x = 0; x < VC; ++x) {
                  uint4* p = reinterpret_cast<uint4*>(g + (x * VK + lo + (idx >> 3)) * 128 + (idx & 7) * 16);
                  uint4 v = *p;
                  if (!finite_words<FP8>(v)) {
                    v.x = finite_word<FP8>(v.x);
                    v.y = finite_word<FP8>(v.y);
                    v.z = finite_word<FP8>(v.z);
                    v.w = finite_word<FP8>(v.w);
                    *p = v;
                  }
                }
              }
              for (int idx = lane; idx < (VK - hi) * 8; idx += 32) {
#pragma unroll
                for (int x = 0; x < VC; ++x)
                  *reinterpret_cast<uint4*>(g + (x * VK + hi + (idx >> 3)) * 128 + (idx & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (el) {
                fence_release_shared();
                mbar_complete_tx_cluster(lb + 8 * slot, kCSlot);   // this CTA's share is in place
              }
            }
            if (++slot == kVRing) {
              slot = 0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          rows = next_rows;
        }
      }
      if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
      }
    } else if (warp == 1) {
      // ================================================================== QK^T (even CTA)
      if (leader) {
        const bool el = elect_one();
        constexpr uint32_t idesc = make_idesc(128, 256, FP8 ? 0u : 1u, 0, 0);
        // Q chunk c (64 columns): [64 rows][128 B] at 8 KB c; E4M3: hi and lo are the first and
        // second 512 bytes of each 1 KB group of 8 rows, 64-byte rows
        const uint64_t dQ0 = make_sdesc(sQ, 16, 1024, FP8 ? kSwizzle64 : kSwizzle128);
        const uint64_t dK0 = make_sdesc(sK, 16, 1024, kSwizzle128);          // [128 keys][128 B]
        uint32_t slot = 0, ph = 0, n = 0, uc = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
          const CUnit U = load_cunit(a, u);
          if (U.te == U.tb) continue;
          ok = wait_issue(b_qfull, uc & 1);
          for (int tile = U.tb; tile < U.te && ok; ++tile, ++n) {
            const uint32_t d = tmem + (n & 1) * 128;
            ok = wait_warp(b_sempty + 8 * (n & 1), ((n >> 1) & 1) ^ 1);
#pragma unroll 1
            for (int c = 0; c < KS && ok; ++c) {
              ok = wait_warp(b_kfull + 8 * slot, ph);
              if (!ok) break;
              tc_fence_after();
              const uint64_t kd = dK0 + (uint64_t)(slot * (kCSlot >> 4));
              if (!el) {
              } else if constexpr (FP8) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  if (c == KS - 1 && kk >= 2) break;       // the row's last 64 bytes
                  const uint64_t qd = dQ0 + (uint64_t)((2 * c + (kk >> 1)) * (kCQChunk >> 4) + (kk & 1) * 2);
                  umma_pair_f8(d, qd, kd + 2 * kk, idesc, (c | kk) != 0);
                  umma_pair_f8(d, qd + (512 >> 4), kd + 2 * kk, idesc, 1u);
                }
              } else {
                const uint64_t qd = dQ0 + (uint64_t)(c * (kCQChunk >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_pair_f16(d, qd + 2 * kk, kd + 2 * kk, idesc, (c | kk) != 0);
              }
              if (el) umma_pair_commit(b_kempty + 8 * slot);
              if (++slot == kKRing) {
                slot = 0;
                ph ^= 1;
              }
            }
            if (!ok) break;
            if (el) {
              umma_pair_commit(b_sfull + 8 * (n & 1));
              if (tile == U.te - 1) umma_pair_commit(b_qempty);
            }
          }
          ++uc;
        }
        // every MMA issued has completed before tensor memory is released
        if (el) umma_pair_commit(b_drain);
        volatile uint32_t no_abort = 0;
        mbar_wait(b_drain, 0, &no_abort, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
      }
    } else if (warp == 3) {
      // ================================================================== PV (even CTA)
      if (leader) {
        const bool el = elect_one();
        constexpr uint32_t idesc = make_idesc(128, 256, FP8 ? 0u : 1u, 0, 1);
        const uint64_t dP0 = make_sdesc(sP, 16, 1024, kSwizzle128);          // [key chunk][64 rows][128 B]
        const uint64_t dV0 = make_sdesc(sV, VK * 128, 1024, kSwizzle128);    // [VC pieces][VK keys][128 B], MN-major
        constexpr int kHalfSlots = kChunkTile / VK / 2;
        uint32_t slot = 0, ph = 0, n = 0, uc = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
          const CUnit U = load_cunit(a, u);
          if (U.te == U.tb) continue;
          for (int tile = U.tb; tile < U.te && ok; ++tile, ++n) {
            const int ns = value_slots<VK>(U.hi, tile);
            if (tile == U.tb) ok = wait_warp(b_oempty, (uc & 1) ^ 1);
            // by halves of the tile's keys, whose P is written and released apart: the way from one
            // PV over its completion, the next P and the signal back is hidden by the other half
#pragma unroll 1
            for (int s = 0; s < kHalfSlots * 2 && ok; ++s) {
              if (s % kHalfSlots == 0) {
                ok = wait_issue(b_p + 8 * (s / kHalfSlots), n & 1);
                if (!ok) break;
              }
              if (s < ns) {
                ok = wait_issue(b_vfull + 8 * slot, ph);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = dV0 + (uint64_t)(slot * (kCSlot >> 4));
                // keys VK s ..: half s & 1 of a 128-byte chunk of P's columns; E4M3: lo 16 KB after hi
                const uint64_t pd = dP0 + (uint64_t)((s >> 1) * (8192 >> 4) + (s & 1) * 4);
                const bool first = tile == U.tb && s == 0;
                if (el) {
#pragma unroll
                  for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                      const uint64_t vk = vd + (uint64_t)((j * 8192 + kk * (FP8 ? 4096 : 2048)) >> 4);
                      const uint32_t acc = !(first && kk == 0);
                      if constexpr (FP8) {
                        umma_pair_f8(tmem + kCOCol + 128 * j, pd + 2 * kk, vk, idesc, acc);
                        umma_pair_f8(tmem + kCOCol + 128 * j, pd + 2 * kk + (16384 >> 4), vk, idesc | kIdescE5M2A, 1u);
                      } else {
                        umma_pair_f16(tmem + kCOCol + 128 * j, pd + 2 * kk, vk, idesc, acc);
                      }
                    }
                  umma_pair_commit(b_vempty + 8 * slot);
                }
                if (++slot == kVRing) {
                  slot = 0;
                  ph ^= 1;
                }
              }
              if (s % kHalfSlots == kHalfSlots - 1 && el) umma_pair_commit(b_pv + 8 * (s / kHalfSlots));
            }
          }
          ++uc;
        }
        if (el) umma_pair_commit(b_drain);
        volatile uint32_t no_abort = 0;
        mbar_wait(b_drain, 0, &no_abort, err, MLA_DEVERR_TIMEOUT, a.wait_limit_ns);
      }
    }
  } else if (warp < 12) {
    // ================================================================== softmax
    regs_lower<112>();
    constexpr uint32_t sbar = 1;
    const int t = threadIdx.x - 128;
    const int row = t & 63, half = (t >> 6) & 1, quarter = t >> 7;   // row of this CTA; keys 128 half + 64 quarter ..
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const float c0 = a.softmax_scale * (FP8 ? __ldg(a.kv_scale) : 1.0f) * kCLog2e;
    uint32_t n = 0, uc = 0, us = 0, xp = 0;
    bool fail = false, stop = false;
    for (int u = u0; u < u1 && !stop; ++u) {
      const CUnit U = load_cunit(a, u);
      const int T = U.te - U.tb;
      const int br = 64 * (int)rank + row;     // row of the block
      int vis = U.hi;
      if (a.causal && br < U.nrows) vis = max(0, U.vis + (U.srow0 + br) / a.H);
      float c = c0;
      if (FP8 && T > 0) {
        fail |= !wait(b_qsc, uc & 1);
        c *= qf_s[row];
        if (named_bar_or(sbar, 256, fail)) break;
        if (t == 0) mbar_arrive(b_qfree);
      }
      float ref = -INFINITY, sum = 0.f;
      float recent = -INFINITY;                // E4M3: this thread's largest score of the window
      if (FP8) top_s[t] = -INFINITY;
      for (int k = 0; k < T; ++k, ++n) {
        const int tile = U.tb + k;
        if (a.test_stall && n == 0) fail |= !wait(b_never, 0);   // tests: this wait runs out
        fail |= !wait(b_sfull + 8 * (n & 1), (n >> 1) & 1);
        tc_fence_after();
        const uint32_t ts = tmem + lane_addr + (n & 1) * 128 + 64 * quarter;
        const int mine = vis - tile * kChunkTile - 128 * half - 64 * quarter;   // keys of this thread its row sees
        // pass 1: the largest score. Scores stay raw (times the sign of their factor) and are scaled
        // after the reference is subtracted, so that the difference of large ones is exact.
        float mx = -INFINITY;
        const bool none = __all_sync(0xffffffffu, mine <= 0);    // no row of the warp sees its keys here
        if (!none) {
          float s[64];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld16(ts + 16 * i, s + 16 * i);
          tmem_wait_ld();
          if (c < 0.f) {
#pragma unroll
            for (int x = 0; x < 64; ++x) s[x] = -s[x];
          }
          if (mine < 64) {
#pragma unroll
            for (int x = 0; x < 64; ++x) s[x] = x < mine ? s[x] : -INFINITY;
          }
          mx = max64(s);
        }
        float alpha = 1.f;
        bool rescale = false, move = k == 0;
        const bool look = FP8 && k % Cfg::kWindow == Cfg::kWindow - 1 && k + 1 < T;
        if (FP8) {
          recent = fmaxf(recent, mx);
          if (look) mx = recent;
        }
        if (!move)
          move = named_bar_or(sbar, 256,
                              fail || (mx > ref && (ref == -INFINITY || (mx - ref) * fabsf(c) > Cfg::kRescaleLog2)) ||
                                  (look && (ref - mx) * fabsf(c) > Cfg::kLowerLog2));
        if (move) {
          mx_s[xp][t] = mx;
          if (named_bar_or(sbar, 256, fail)) { stop = true; break; }
          const float* m = mx_s[xp];
          const float rm = fmaxf(fmaxf(mx, m[t ^ 64]), fmaxf(m[t ^ 128], m[t ^ 192]));
          float nm = look && (rm - ref) * fabsf(c) <= Cfg::kRescaleLog2 ? ref : fmaxf(ref, rm);
          xp ^= 1;
          if (look && rm != -INFINITY && (ref - rm) * fabsf(c) > Cfg::kLowerLog2)
            nm = fminf(ref, fmaxf(rm, top_s[t] - Cfg::kSpanLog2 / fabsf(c)));
          alpha = ref == -INFINITY ? 0.f : ex2_approx((ref - nm) * fabsf(c));   // none seen before: O and sum are 0
          rescale = k > 0;
          if (look) rescale = named_bar_or(sbar, 256, nm != ref);   // a thread's quarter may be low, its row not
          ref = nm;
          if (FP8) top_s[t] = fmaxf(top_s[t], ref);
          sum *= alpha;
        }
        if (look) recent = -INFINITY;
        // pass 2: P, packed
        const float off = ref == -INFINITY ? 0.f : c < 0.f ? ref : -ref;
        uint32_t pw[32];        // bf16: key pairs; E4M3: hi bytes (words 0-15), lo bytes (16-31)
        if (none) {
#pragma unroll
          for (int x = 0; x < 32; ++x) pw[x] = 0u;
        } else
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float s[32];
          tmem_ld32(ts + 32 * i, s);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            add2(s[x], s[x + 1], off, off);
            fma2(s[x], s[x + 1], c, Cfg::kPOffLog2);
          }
          if (mine < 32 * i + 32) {
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = 32 * i + x < mine ? s[x] : -INFINITY;
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) s[x] = ex2_approx(s[x]);
          sum += sum32(s);                               // the normaliser sums the unrounded values
          if constexpr (FP8) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const uint32_t o0 = split_e4m3_e5m2x2(s[4 * x], s[4 * x + 1]);
              const uint32_t o1 = split_e4m3_e5m2x2(s[4 * x + 2], s[4 * x + 3]);
              pw[8 * i + x] = __byte_perm(o0, o1, 0x5410);
              pw[16 + 8 * i + x] = __byte_perm(o0, o1, 0x7632);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              __nv_bfloat162 h = __floats2bfloat162_rn(s[2 * x], s[2 * x + 1]);
              pw[16 * i + x] = *reinterpret_cast<uint32_t*>(&h);
            }
          }
        }
        // S has been read: its buffer is free (nothing this thread wrote is published with it)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(lead(b_sempty + 8 * (n & 1)));
        // this half of P is free once the previous tile's PV over it has completed, O once all of it
        if (n > 0) {
          fail |= !wait(b_pv + 8 * half, (n - 1) & 1);
          if (rescale) fail |= !wait(b_pv + 8 * (half ^ 1), (n - 1) & 1);
        }
        if (rescale) {
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            float o[16];
            const uint32_t ta = tmem + lane_addr + kCOCol + 128 * quarter + 16 * cc;
            tmem_ld16(ta, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(ta, o);
          }
          tmem_wait_st();
          tc_fence_before();
          named_bar_sync(sbar, 256);             // all of O, before either half of P is announced
        }
        if constexpr (FP8) {
          // hi and lo (16 KB on): 64 bytes of the row of 128-key chunk `half`
          uint8_t* p = gP + half * 8192 + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *reinterpret_cast<uint4*>(p + h * 16384 + (((4 * quarter + x) ^ (row & 7)) << 4)) =
                  make_uint4(pw[16 * h + 4 * x], pw[16 * h + 4 * x + 1], pw[16 * h + 4 * x + 2], pw[16 * h + 4 * x + 3]);
        } else {
          // the row of 64-key chunk 2 half + quarter
          uint8_t* p = gP + (2 * half + quarter) * 8192 + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4*>(p + ((x ^ (row & 7)) << 4)) =
                make_uint4(pw[4 * x], pw[4 * x + 1], pw[4 * x + 2], pw[4 * x + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        // a failed wait is carried to the next barrier of all 256 threads
        fail |= named_bar_or(4 + half, 128, fail);
        if (!fail && (t & 191) == 0) {
          if (leader) {
            mbar_arrive(b_p + 8 * half);
          } else {
            fence_release_shared();
            mbar_arrive_cluster_relaxed(lead(b_p + 8 * half));
          }
        }
      }
      if (stop) break;
      // the row's reference and this thread's sum, for the epilogue
      if (us > 0) fail |= !wait(b_statfree, (us - 1) & 1);
      sum_s[t] = sum;
      if (t < 128) ref_s[t] = ref == -INFINITY ? ref : ref * fabsf(c);
      mbar_arrive(b_stat);
      ++us;
      if (T > 0) ++uc;
    }
  } else {
    // ================================================================== q terms, epilogue
    regs_raise<216>();
    constexpr uint32_t ebar = 2;
    const int t = threadIdx.x - 384;
    const int row = t & 63, half = t >> 6;     // epilogue: this thread's row and value columns 256 half ..
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const float kvs = FP8 ? __ldg(a.kv_scale) : 1.0f;
    uint32_t n = 0, us = 0, uq = 0;
    bool fail = false;
    // E4M3: the 64 rows of this CTA, bf16 as TMA landed them, become q' = q 2^e (the row's largest
    // |q| in [128, 256)) as E4M3 hi and lo in place: every 1 KB group of 8 rows x 64 columns becomes
    // hi in its first 512 bytes and lo in its second (64-byte swizzled rows). A warp owns whole
    // groups; lane 4 q + p holds 16-byte units p and p + 4 of row q. False after a failed wait.
    auto split_q = [&]() -> bool {
      bool mine = wait(b_qraw, uq & 1);
      if (mine && uq > 0) mine = wait(b_qfree, (uq - 1) & 1);   // the previous factors were read
      if (named_bar_or(ebar, 128, !mine)) return false;
      const int qrow = lane >> 2, part = lane & 3;
#pragma unroll 1
      for (int g = warp - 12; g < 8; g += 4) {
        auto block_of = [&](int c) -> uint8_t* { return gQ + c * kCQChunk + g * 1024; };
        __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int c = 0; c < 9; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = *reinterpret_cast<const uint4*>(block_of(c) + qrow * 128 + (((part + 4 * h) ^ qrow) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[k])));
          }
        float mx = fmaxf(__low2float(m2), __high2float(m2));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int e = 0;
        if (mx > 0.f) e = min(max(7 - ((int)((__float_as_uint(mx) >> 23) & 0xFFu) - 127), -126), 126);
        const float f = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll 1
        for (int c = 0; c < 9; ++c) {
          uint8_t* blk = block_of(c);
          uint4 v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[h] = *reinterpret_cast<const uint4*>(blk + qrow * 128 + (((part + 4 * h) ^ qrow) << 4));
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int un = part + 4 * h;           // columns 8 un .. of the chunk
            const uint32_t w[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = split_e4m3x2(bf_lo(w[k]) * f, bf_hi(w[k]) * f);
            const uint32_t off = qrow * 64 + (((un >> 1) ^ ((qrow >> 1) & 3)) << 4) + (un & 1) * 8;
            *reinterpret_cast<uint2*>(blk + off) = make_uint2(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410));
            *reinterpret_cast<uint2*>(blk + 512 + off) =
                make_uint2(__byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
          }
        }
        if (part == 0) qf_s[8 * g + qrow] = __uint_as_float((uint32_t)(127 - e) << 23);
      }
      fence_proxy_async_smem();
      named_bar_sync(ebar, 128);
      if (t == 0) {
        mbar_arrive(b_qsc);
        // the issuer needs both CTAs' terms
        if (leader) {
          mbar_arrive(b_qfull);
        } else {
          fence_release_shared();
          mbar_arrive_cluster_relaxed(lead(b_qfull));
        }
      }
      ++uq;
      return true;
    };
    // E4M3: q of the first unit before anything else, then before a unit's results q of the next
    // one, whose load waits for the unit's QK^T only (one loop, so that the split is there once)
    int nu = u0;                               // the next unit whose q may have to be split
    for (int u = FP8 ? u0 - 1 : u0; u < u1; ++u) {
      const CUnit U = load_cunit(a, max(u, u0));
      const int T = U.te - U.tb;
      if (FP8 && (u < u0 || T > 0)) {
        bool found = false;
        for (; nu < u1 && !found; ++nu) {
          const CUnit N = load_cunit(a, nu);
          found = N.te != N.tb;
        }
        if (found && !split_q()) break;
      }
      if (u < u0) continue;
      n += T;
      fail |= !wait(b_stat, us & 1);
      const float ref = ref_s[t], sum = (sum_s[t] + sum_s[t ^ 64]) + (sum_s[t + 128] + sum_s[(t ^ 64) + 128]);
      mbar_arrive(b_statfree);
      ++us;
      if (T > 0) fail |= !wait(b_pv + 8, (n - 1) & 1);
      if (named_bar_or(ebar, 128, fail)) break;
      tc_fence_after();
      const int br = 64 * (int)rank + row;
      const bool keep = br < U.nrows;
      const float inv = sum == 0.f ? 0.f : kvs / sum;          // a row that sees no key: zeros
      const int64_t orow = (int64_t)U.row0 + br;
      const int odd = lane & 1;
      const bool keep0 = br - odd < U.nrows, keep1 = br - odd + 1 < U.nrows;   // the pair's rows
      auto load_o = [&](int i, float* o) {       // 32 columns, normalised
        if (T > 0) {
          tmem_ld32(tmem + lane_addr + kCOCol + 32 * i, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] *= inv;         // a row that sees no key has O = 0
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        }
      };
      // O has been read: the next unit's first PV may overwrite it
      auto release_o = [&]() {
        if (T == 0) return;
        tc_fence_before();
        named_bar_sync(ebar, 128);
        if (t == 0) {
          if (leader) mbar_arrive(b_oempty);
          else mbar_arrive_cluster_relaxed(lead(b_oempty));
        }
      };
      if (U.slot < 0) {
        // all of the thread's columns into registers as bf16 first, so that the next unit's PV
        // waits for the reads and not for the stores
        uint32_t w[128];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float o[32];
          load_o(i, o);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * x], o[2 * x + 1]);
            w[16 * i + x] = *reinterpret_cast<uint32_t*>(&h);
          }
        }
        release_o();
        uint8_t* p = reinterpret_cast<uint8_t*>(a.out + (orow - odd) * kDV + 256 * half) + 32 * odd;
#pragma unroll
        for (int x = 0; x < 8; ++x) store_pair64(p + 64 * x, kDV * 2, w + 16 * x, odd, keep0, keep1, a.out_wide != 0);
      } else {
        uint8_t* p = reinterpret_cast<uint8_t*>(a.part_o + ((int64_t)U.slot * kChunkRows + br - odd) * kDV + 256 * half) + 32 * odd;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          float o[32];
          load_o(i, o);
          uint32_t w[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) w[x] = __float_as_uint(o[x]);
#pragma unroll
          for (int x = 0; x < 2; ++x) store_pair64(p + 128 * i + 64 * x, kDV * 4, w + 16 * x, odd, keep0, keep1, true);
        }
        release_o();
      }
      if (half == 0 && keep) {
        // P was computed times 2^kPOffLog2, and so was the row sum
        const float l = sum == 0.f ? -INFINITY : (ref + log2f(sum) - Cfg::kPOffLog2) * kCLn2;
        if (U.slot < 0) a.lse[orow] = l;
        else a.part_lse[(int64_t)U.slot * kChunkRows + br] = l;
      }
    }
  }

  // ==================================================================== teardown
  tc_fence_before();
  __syncthreads();
  cluster_sync();                         // neither CTA leaves while its peer may still use it
  tc_fence_after();
  if (warp == 0) tmem_dealloc_pair(tmem, kCTmemCols);
}

namespace {

template <bool FP8, bool kSub>
cudaError_t prepare_variant() {
  cudaError_t e =
      cudaFuncSetAttribute(chunk_kernel<FP8, kSub>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCDynBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, chunk_kernel<FP8, kSub>);
  if (e != cudaSuccess) return e;
  return (int)attr.sharedSizeBytes > kCStaticBudget ? cudaErrorInvalidConfiguration : cudaSuccess;
}

}  // namespace

cudaError_t chunk_prepare(bool fp8) {
  cudaError_t e = fp8 ? prepare_variant<true, false>() : prepare_variant<false, false>();
  if (e != cudaSuccess) return e;
  return fp8 ? prepare_variant<true, true>() : prepare_variant<false, true>();
}

cudaError_t launch_chunk(const ChunkArgs& a, bool fp8, int pairs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kCThreads);
  cfg.dynamicSmemBytes = kCDynBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // overlap the scheduler
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // pages that are no multiple of 64 rows take the kernel that loads a slot as several boxes
  const bool sub = a.k_box < 64;
  if (fp8) return sub ? cudaLaunchKernelEx(&cfg, chunk_kernel<true, true>, a) : cudaLaunchKernelEx(&cfg, chunk_kernel<true, false>, a);
  return sub ? cudaLaunchKernelEx(&cfg, chunk_kernel<false, true>, a) : cudaLaunchKernelEx(&cfg, chunk_kernel<false, false>, a);
}

}  // namespace mla
