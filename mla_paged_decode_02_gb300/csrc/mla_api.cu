// mla_api.cu — the C ABI (include/mla.h): argument checks, workspace layout, TMA
// descriptors and the launch sequence  schedule -> decode -> combine  on one stream.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>
#include <vector>
#include <cudaTypedefs.h>
#include "mla_chunk.h"
#include "mla_index.h"
#include "mla_internal.h"
#include "mla_ptx.cuh"
#include "mla_rope.h"
#include "../../include/mla.h"

#define MLA_EXPORT extern "C" __attribute__((visibility("default")))

namespace mla {
namespace {

constexpr int kMaxDevices = 64;

std::atomic<int> g_num_sms[kMaxDevices];
std::atomic<uint32_t> g_prepared[kMaxDevices];   // bit per decode variant
std::mutex g_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// decode-kernel timing window (mla_profile_begin / mla_profile_end)
struct ProfileWindow {
  std::vector<cudaEvent_t> ev;   // 2 per launch: before, after
  int cap = 0, next = 0;
  bool on = false;
};
ProfileWindow g_prof;
constexpr int kMaxProfiledLaunches = 4096;

// test hooks (mla_test_set_hooks): the wait bound passed to the kernels and the stall flag
std::atomic<uint64_t> g_wait_limit_ns{kWaitLimitNs};
std::atomic<int32_t> g_test_stall{0};

int variant_bit(int rc, bool fp8) {
  return (rc == 16 ? 0 : rc == 32 ? 2 : rc == 64 ? 4 : 6) + (fp8 ? 1 : 0);
}

cudaError_t current_device(int* dev) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= kMaxDevices) return cudaErrorInvalidDevice;
  return cudaSuccess;
}

int sm_count(int dev) {
  int n = g_num_sms[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return -1;
  g_num_sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool get_encoder() {
  if (g_encode) return true;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_encode) return true;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr)
    return false;
  g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return true;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

mla_status check_params(const mla_decode_params* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->s_q < 1 || p->num_heads < 1 || p->page_size < 1 || p->num_pages < 1 ||
      p->max_blocks_per_seq < 1 || p->max_seq_len < 1)
    return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (p->causal != 0 && p->causal != 1) return MLA_ERR_INVALID_ARG;
  if (p->max_seq_len < p->s_q) return MLA_ERR_INVALID_ARG;
  if (p->page_size % 8 != 0 || p->page_size > 1024) return MLA_ERR_UNSUPPORTED;
  if (p->s_q > kMaxSq || (int64_t)p->s_q * p->num_heads > kMaxRows) return MLA_ERR_UNSUPPORTED;
  if (p->batch > kMaxBatch || p->max_seq_len > kMaxSeqLen) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->num_pages * p->page_size >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->max_blocks_per_seq * p->page_size < p->s_q) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

// The cache as [rows / 8 groups][9 chunks][8 rows][64 elements] (strides 8 rows, one
// chunk, one row): a box of `chunks` chunks x box_rows / 8 groups lands in shared memory
// as [group][chunk][8 rows][64 elements]. bf16 rows (128 B) are 128-byte swizzled for
// the MMA. E4M3 rows (64 B) with sw64 are 64-byte swizzled: the layout of the 8-bit MMA
// operands (CTA pairs), and one in which 32 threads reading one key row each hit distinct
// banks (the converting threads of the single-CTA kernel); its E4M3 value rows are plain.
bool encode_kv_map(CUtensorMap* m, const void* cache, int64_t rows, uint32_t chunks, uint32_t box_rows,
                   bool fp8, bool sw64) {
  const cuuint64_t es = fp8 ? 1 : 2;
  cuuint64_t dims[4] = {64, 8, 9, (cuuint64_t)(rows / 8)};
  cuuint64_t strides[3] = {kDQK * es, 64 * es, kDQK * es * 8};
  cuuint32_t box[4] = {64, 8, chunks, box_rows / 8};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        !fp8 ? CU_TENSOR_MAP_SWIZZLE_128B
                             : sw64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// q as [B][R/8 groups][9 chunks][8 rows][64 elements]: a box of 8 groups x 9 chunks is 64
// whole 1152-byte rows (one contiguous piece each, the cheapest for TMA), landing as
// [group][chunk][8 rows][64] with 128-byte swizzle. Needs R % 8 == 0.
bool encode_q_rows_map(CUtensorMap* m, const void* q, int B, int R) {
  cuuint64_t dims[5] = {64, 8, 9, (cuuint64_t)(R / 8), (cuuint64_t)B};
  cuuint64_t strides[4] = {(cuuint64_t)kDQK * 2, 128, (cuuint64_t)kDQK * 2 * 8, (cuuint64_t)kDQK * 2 * R};
  cuuint32_t box[5] = {64, 8, 9, 8, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(q), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_q_map(CUtensorMap* m, const void* q, int B, int R, int rc) {
  cuuint64_t dims[3] = {(cuuint64_t)kDQK, (cuuint64_t)R, (cuuint64_t)B};
  cuuint64_t strides[2] = {(cuuint64_t)kDQK * 2, (cuuint64_t)kDQK * 2 * R};
  cuuint32_t box[3] = {64, (cuuint32_t)rc, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                        box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace
}  // namespace mla

using namespace mla;

MLA_EXPORT int32_t mla_abi_version(void) { return MLA_ABI_VERSION; }

MLA_EXPORT const char* mla_status_string(int32_t s) {
  switch (s) {
    case MLA_OK: return "ok";
    case MLA_ERR_INVALID_ARG: return "invalid argument";
    case MLA_ERR_UNSUPPORTED: return "unsupported configuration";
    case MLA_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case MLA_ERR_CUDA: return "CUDA runtime error";
    case MLA_ERR_TIMEOUT: return "device pipeline wait timed out";
    case MLA_ERR_DEVICE_INDEX: return "device-side index or length out of range";
    default: return "unknown status";
  }
}

MLA_EXPORT size_t mla_decode_workspace_size(const mla_decode_params* p, int32_t num_sms) {
  if (check_params(p) != MLA_OK) return 0;
  if (num_sms <= 0) {
    int dev;
    if (current_device(&dev) != cudaSuccess) return 0;
    num_sms = sm_count(dev);
    if (num_sms <= 0) return 0;
  }
  const Plan plan = make_plan(p->s_q * p->num_heads, p->kv_dtype == MLA_KV_FP8_E4M3);
  return ws_layout(p->batch, plan, plan_workers(plan, num_sms)).total;
}

namespace mla {
namespace {
// The step's new tokens for the fused cache write (num == 0: none).
struct FusedWrite {
  const void* latent;
  const void* rope;
  const int64_t* slots;
  int32_t num;
};
}  // namespace
}  // namespace mla

static mla_status decode_impl(const mla_decode_params* p, const void* q, const void* kv_cache,
                              const int32_t* block_table, const int32_t* seq_lens, float softmax_scale,
                              const float* kv_scale, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, mla_stream_t stream, const FusedWrite& fw) {
  mla_status st = check_params(p);
  if (st != MLA_OK) return st;
  const bool fp8 = p->kv_dtype == MLA_KV_FP8_E4M3;
  if (!q || !kv_cache || !block_table || !seq_lens || !out || !lse || !workspace)
    return MLA_ERR_INVALID_ARG;
  if (fp8 && !kv_scale) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || softmax_scale > 3.0e38f || softmax_scale < -3.0e38f)
    return MLA_ERR_INVALID_ARG;

  int dev;
  if (current_device(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  const int nsm = sm_count(dev);
  if (nsm <= 0) return MLA_ERR_CUDA;
  const int B = p->batch, R = p->s_q * p->num_heads;
  const Plan plan = make_plan(R, fp8);
  const int rc = plan.rc, G = plan.G;
  const int grid = plan_workers(plan, nsm);
  if (grid < 1) return MLA_ERR_UNSUPPORTED;
  const WsLayout w = ws_layout(B, plan, grid);
  if (workspace_bytes < w.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!get_encoder()) return MLA_ERR_CUDA;

  const uint32_t bit = 1u << variant_bit(rc, fp8);
  if (!(g_prepared[dev].load() & bit)) {
    if ((plan.pair ? decode_pair_prepare(fp8) : decode_prepare(rc, fp8)) != cudaSuccess) return MLA_ERR_CUDA;
    g_prepared[dev].fetch_or(bit);
  }

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* hdr = reinterpret_cast<uint32_t*>(ws);
  int4* batch_info = reinterpret_cast<int4*>(ws + w.batch_off);
  int32_t* cta_first = reinterpret_cast<int32_t*>(ws + w.cta_off);
  int4* split_list = reinterpret_cast<int4*>(ws + w.split_off);
  int4* units = reinterpret_cast<int4*>(ws + w.units_off);
  float* plse = reinterpret_cast<float*>(ws + w.plse_off);
  float* po = reinterpret_cast<float*>(ws + w.po_off);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  SchedArgs sa{};
  sa.seq_lens = seq_lens;
  sa.hdr = hdr;
  sa.batch_info = batch_info;
  sa.cta_first = cta_first;
  sa.split_list = split_list;
  sa.units = units;
  sa.B = B;
  sa.s_q = p->s_q;
  sa.G = G;
  const int64_t cap = (int64_t)p->max_blocks_per_seq * p->page_size;
  sa.max_len = (int)(cap < p->max_seq_len ? cap : p->max_seq_len);
  sa.grid = grid;
  sa.tile = plan.tile;
  // a unit's set-up (its q, the pipeline's refill, its epilogue) is charged to the CTA that
  // starts the stream, in tiles of streaming: measured best at 2 for bf16 CTA pairs, 3 for
  // FP8 pairs and 4 for the FP8 cache with up to 64 rows; with bf16 and up to 64 rows a unit
  // change costs little (0)
  sa.setup = plan.pair ? (fp8 ? 3 : 2) : fp8 ? 4 : 0;
  sa.max_units = w.max_units;
  sa.max_split = w.max_split;
  sa.max_slots = w.max_slots;
  if (fw.num > 0) {
    // the new tokens' rows go into the cache ahead of the decode: CTAs of the scheduler's
    // launch write them next to the schedule computation (for very large writes, the
    // cache-write kernel runs ahead of the scheduler instead)
    const int64_t total_slots = (int64_t)p->num_pages * p->page_size;
    if (fw.num <= kMaxFusedWriteTokens) {
      sa.w_latent = static_cast<const uint4*>(fw.latent);
      sa.w_rope = static_cast<const uint4*>(fw.rope);
      sa.w_slots = fw.slots;
      sa.w_cache = static_cast<uint8_t*>(const_cast<void*>(kv_cache));
      sa.w_kv_scale = kv_scale;
      sa.w_total_slots = total_slots;
      sa.w_n = fw.num;
      sa.w_fp8 = fp8 ? 1 : 0;
    } else if (launch_cache_write(fw.latent, fw.rope, fw.slots, fw.num, const_cast<void*>(kv_cache), total_slots, fp8,
                                  kv_scale, nullptr, s) != cudaSuccess) {
      return MLA_ERR_CUDA;
    }
  }
  if (launch_schedule(sa, s) != cudaSuccess) return MLA_ERR_CUDA;

  DecodeArgs da;
  std::memset(&da, 0, sizeof(da));
  // key / value boxes of gcd(P, 64) rows never straddle a page
  const int box_rows = std::min(64, p->page_size & -p->page_size);
  // a CTA of a pair holds 64 of its unit's 128 rows (as whole rows when R % 8 == 0)
  da.q_whole_rows = plan.pair && R % 8 == 0 ? 1 : 0;
  if (da.q_whole_rows ? !encode_q_rows_map(&da.tm_q, q, B, R) : !encode_q_map(&da.tm_q, q, B, R, plan.pair ? 64 : rc))
    return MLA_ERR_INVALID_ARG;
  {
    const int64_t rows = (int64_t)p->num_pages * p->page_size;
    // chunks per key / value box: a pair loads 256-byte pieces of each bf16 key row (2
    // chunks) or whole E4M3 key rows (9 chunks), and 4 adjacent chunks of each value row
    const uint32_t kc = plan.pair ? (fp8 ? 9u : 2u) : (uint32_t)decode_key_chunks_per_slot(rc, fp8);
    const uint32_t vc = plan.pair ? 4u : (uint32_t)decode_value_chunks_per_box(rc, fp8);
    // E4M3 keys and values are 64-byte swizzled: the MMAs read them as they land
    if (!encode_kv_map(&da.tm_k, kv_cache, rows, kc, (uint32_t)box_rows, fp8, true) ||
        !encode_kv_map(&da.tm_v, kv_cache, rows, vc, (uint32_t)box_rows, fp8, true))
      return MLA_ERR_INVALID_ARG;
  }
  da.kv_cache = kv_cache;
  da.block_table = block_table;
  da.batch_info = batch_info;
  da.units = units;
  da.cta_first = cta_first;
  da.hdr = hdr;
  da.out = static_cast<__nv_bfloat16*>(out);
  da.lse = lse;
  da.part_o = po;
  da.part_lse = plse;
  da.err = hdr;
  da.kv_scale = kv_scale;
  da.s_q = p->s_q;
  da.H = p->num_heads;
  da.R = R;
  da.P = p->page_size;
  da.box_rows = box_rows;
  da.MB = p->max_blocks_per_seq;
  da.num_pages = p->num_pages;
  da.causal = p->causal;
  da.softmax_scale = softmax_scale;
  da.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  da.test_stall = g_test_stall.load(std::memory_order_relaxed);
  const bool timed = g_prof.on && g_prof.next < g_prof.cap;
  if (timed && cudaEventRecord(g_prof.ev[2 * g_prof.next], s) != cudaSuccess) return MLA_ERR_CUDA;
  const cudaError_t le = plan.pair ? launch_decode_pair(da, fp8, grid, s) : launch_decode(da, rc, fp8, grid, s);
  if (le != cudaSuccess) return MLA_ERR_CUDA;
  if (timed) {
    if (cudaEventRecord(g_prof.ev[2 * g_prof.next + 1], s) != cudaSuccess) return MLA_ERR_CUDA;
    ++g_prof.next;
  }

  CombineArgs ca{};
  ca.hdr = hdr;
  ca.err = hdr;
  ca.w_slots = fw.num > 0 ? fw.slots : nullptr;
  ca.w_n = fw.num;
  ca.w_total_slots = (int64_t)p->num_pages * p->page_size;
  ca.block_table = block_table;
  ca.batch_info = batch_info;
  ca.B = p->batch;
  ca.MB = p->max_blocks_per_seq;
  ca.P = p->page_size;
  ca.num_pages = p->num_pages;
  ca.split_list = split_list;
  ca.part_o = po;
  ca.part_lse = plse;
  ca.out = static_cast<__nv_bfloat16*>(out);
  ca.lse = lse;
  ca.R = R;
  ca.RC = rc;
  // up to 2 * workers cut streams x RC rows: 8 * #SM blocks of 8 warps give every (stream,
  // row) task its own warp for RC <= 32 and at most two rounds for RC = 64 or 128 (the
  // combine is a few dependent global loads per task: latency, not bandwidth)
  if (launch_combine(ca, 8 * nsm, s) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

MLA_EXPORT mla_status mla_test_set_hooks(uint64_t wait_limit_ns, int32_t stall) {
  if (stall != 0 && stall != 1) return MLA_ERR_INVALID_ARG;
  mla::g_wait_limit_ns.store(wait_limit_ns == 0 ? mla::kWaitLimitNs : wait_limit_ns);
  mla::g_test_stall.store(stall);
  return MLA_OK;
}

MLA_EXPORT mla_status mla_decode(const mla_decode_params* p, const void* q, const void* kv_cache,
                                 const int32_t* block_table, const int32_t* seq_lens,
                                 float softmax_scale, const float* kv_scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  return decode_impl(p, q, kv_cache, block_table, seq_lens, softmax_scale, kv_scale, out, lse, workspace,
                     workspace_bytes, stream, FusedWrite{nullptr, nullptr, nullptr, 0});
}

MLA_EXPORT mla_status mla_decode_with_cache_write(const mla_decode_params* p, const void* latent,
                                                  const void* rope, const int64_t* slot_mapping,
                                                  int32_t num_tokens, const void* q, void* kv_cache,
                                                  const int32_t* block_table, const int32_t* seq_lens,
                                                  float softmax_scale, const float* kv_scale, void* out,
                                                  float* lse, void* workspace, size_t workspace_bytes,
                                                  mla_stream_t stream) {
  if (num_tokens < 0) return MLA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!latent || !rope || !slot_mapping)) return MLA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(slot_mapping, 8)))
    return MLA_ERR_INVALID_ARG;
  return decode_impl(p, q, kv_cache, block_table, seq_lens, softmax_scale, kv_scale, out, lse, workspace,
                     workspace_bytes, stream, FusedWrite{latent, rope, slot_mapping, num_tokens});
}

MLA_EXPORT mla_status mla_profile_begin(int32_t max_launches) {
  using mla::g_prof;
  if (max_launches < 1 || max_launches > mla::kMaxProfiledLaunches) return MLA_ERR_INVALID_ARG;
  while ((int)g_prof.ev.size() < 2 * max_launches) {
    cudaEvent_t e;
    if (cudaEventCreate(&e) != cudaSuccess) return MLA_ERR_CUDA;
    g_prof.ev.push_back(e);
  }
  g_prof.cap = max_launches;
  g_prof.next = 0;
  g_prof.on = true;
  return MLA_OK;
}

MLA_EXPORT mla_status mla_profile_end(double* total_ms, int32_t* launches) {
  using mla::g_prof;
  if (total_ms == nullptr || launches == nullptr) return MLA_ERR_INVALID_ARG;
  const int n = g_prof.on ? g_prof.next : 0;
  g_prof.on = false;
  double sum = 0.0;
  for (int i = 0; i < n; ++i) {
    float ms = 0.f;
    if (cudaEventSynchronize(g_prof.ev[2 * i + 1]) != cudaSuccess ||
        cudaEventElapsedTime(&ms, g_prof.ev[2 * i], g_prof.ev[2 * i + 1]) != cudaSuccess)
      return MLA_ERR_CUDA;
    sum += ms;
  }
  *total_ms = sum;
  *launches = n;
  return MLA_OK;
}

MLA_EXPORT mla_status mla_decode_check(const void* workspace, mla_stream_t stream, uint32_t* bits) {
  if (workspace == nullptr) return MLA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return MLA_ERR_CUDA;
  uint32_t word = 0;
  if (cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (bits) *bits = word;
  if (word & MLA_DEVERR_TIMEOUT) return MLA_ERR_TIMEOUT;
  if (word) return MLA_ERR_DEVICE_INDEX;
  return MLA_OK;
}

MLA_EXPORT mla_status mla_cache_write(const void* latent, const void* rope,
                                      const int64_t* slot_mapping, int32_t num_tokens,
                                      void* kv_cache, int32_t num_pages, int32_t page_size,
                                      int32_t kv_dtype, const float* kv_scale,
                                      uint32_t* device_error, mla_stream_t stream) {
  if (num_tokens < 0 || num_pages < 1 || page_size < 1) return MLA_ERR_INVALID_ARG;
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == MLA_KV_FP8_E4M3;
  if (num_tokens == 0) return MLA_OK;
  if (!latent || !rope || !slot_mapping || !kv_cache) return MLA_ERR_INVALID_ARG;
  if (fp8 && !kv_scale) return MLA_ERR_INVALID_ARG;
  if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8) || (device_error && !aligned(device_error, 4)))
    return MLA_ERR_INVALID_ARG;
  const int64_t total = (int64_t)num_pages * page_size;
  if (launch_cache_write(latent, rope, slot_mapping, num_tokens, kv_cache, total, fp8, kv_scale,
                         device_error, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

// ---------------------------------------------------------------- ragged chunk attention
namespace mla {
namespace {

std::atomic<uint32_t> g_chunk_prepared[kMaxDevices];   // bit per cache type

mla_status check_chunk_params(const mla_chunk_params* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_tokens < 0 || p->num_heads < 1 || p->page_size < 1 || p->num_pages < 1 ||
      p->max_blocks_per_seq < 1 || p->max_seq_len < 1)
    return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (p->causal != 0 && p->causal != 1) return MLA_ERR_INVALID_ARG;
  if (p->page_size % 8 != 0 || p->page_size > 1024) return MLA_ERR_UNSUPPORTED;
  if (p->batch > kMaxBatch || p->max_seq_len > kMaxSeqLen || p->num_heads > kMaxRows) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->num_tokens * p->num_heads > kMaxChunkRows) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->num_pages * p->page_size >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// rows of one box: the largest power of two that divides the page, at most `most`
int box_rows_of(int page_size, int most) { return std::min(most, page_size & -page_size); }

bool encode_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return g_encode(m, type, rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of 576 bf16 as [9 chunks][rows][64]
bool encode_rows_map(CUtensorMap* m, const void* base, int64_t rows, uint32_t box_rows, uint32_t chunks) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, 9};
  const cuuint64_t strides[2] = {kDQK * 2, 128};
  const cuuint32_t box[3] = {64, box_rows, chunks};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box);
}
// rows of 576 bytes; columns past the row read as zeros
bool encode_bytes_map(CUtensorMap* m, const void* base, int64_t rows, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)kDQK, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kDQK};
  const cuuint32_t box[2] = {128, box_rows};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box);
}

// the workspace's part of the scheduler's arguments, and the set-up charge of a block
ChunkSchedArgs chunk_sched_args(uint8_t* ws, const ChunkWs& w, int H, int tokens, int pairs, bool fp8) {
  ChunkSchedArgs sa{};
  sa.hdr = reinterpret_cast<uint32_t*>(ws);
  sa.gbase = reinterpret_cast<int32_t*>(ws + w.gbase_off);
  sa.cta_first = reinterpret_cast<int32_t*>(ws + w.cta_off);
  sa.split_list = reinterpret_cast<int4*>(ws + w.split_off);
  sa.units = reinterpret_cast<ChunkUnit*>(ws + w.units_off);
  sa.H = H;
  sa.workers = pairs;
  // a block's set-up (its q, the softmax before the first PV, its results) costs about 0.6 tiles
  // with the bf16 cache, more with E4M3, whose q is split first; prompts of 150 to 2000 tokens
  // with 16 heads: 226, 179, 188 us for 0, 1, 2 (bf16), 324, 227 to 273, 206 to 217, 212 to 258 for
  // 0, 1, 2, 3 (E4M3; the mixed step 99, 99, 98, 99, single tokens alone 64, 61, 63, 64)
  sa.setup = fp8 ? 2 : 1;
  sa.tokens = tokens;
  return sa;
}

// the geometry of a pool of num_pages pages of page_size rows, and its tensor maps
bool encode_chunk_maps(ChunkArgs* ca, const void* q, int tokens, int H, const void* kv_cache, int num_pages, int page_size,
                       bool fp8) {
  const int64_t rows = (int64_t)num_pages * page_size;
  ca->k_box = box_rows_of(page_size, 64);
  ca->v_box = box_rows_of(page_size, fp8 ? 64 : 32);
  ca->H = H;
  ca->P = page_size;
  ca->num_pages = num_pages;
  ca->total_rows = (int32_t)rows;
  return encode_rows_map(&ca->tm_q, q, (int64_t)tokens * H, 64, 9) &&
         (fp8 ? encode_bytes_map(&ca->tm_k, kv_cache, rows, ca->k_box) && encode_bytes_map(&ca->tm_v, kv_cache, rows, ca->v_box)
              : encode_rows_map(&ca->tm_k, kv_cache, rows, ca->k_box, 1) &&
                    encode_rows_map(&ca->tm_v, kv_cache, rows, ca->v_box, ca->k_box < 64 ? 1 : 4));
}

// the attention kernel over the units that `sa` names, and the merge of the blocks it cut
mla_status launch_chunk_pair(ChunkArgs& ca, ChunkCombineArgs& cc, const ChunkSchedArgs& sa, uint8_t* ws, const ChunkWs& w,
                             float softmax_scale, const float* kv_scale, void* out, float* lse, bool fp8, int pairs,
                             int merge_blocks, cudaStream_t s) {
  ca.units = sa.units;
  ca.cta_first = sa.cta_first;
  ca.err = sa.hdr;
  ca.out = static_cast<__nv_bfloat16*>(out);
  ca.out_wide = aligned(out, 32) ? 1 : 0;
  ca.lse = lse;
  ca.part_o = reinterpret_cast<float*>(ws + w.po_off);
  ca.part_lse = reinterpret_cast<float*>(ws + w.plse_off);
  ca.kv_scale = kv_scale;
  ca.softmax_scale = softmax_scale;
  ca.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  ca.test_stall = g_test_stall.load(std::memory_order_relaxed);
  if (launch_chunk(ca, fp8, pairs, s) != cudaSuccess) return MLA_ERR_CUDA;
  cc.hdr = sa.hdr;
  cc.err = sa.hdr;
  cc.split_list = sa.split_list;
  cc.part_o = ca.part_o;
  cc.part_lse = ca.part_lse;
  cc.out = ca.out;
  cc.lse = ca.lse;
  if (launch_chunk_combine(cc, kChunkRows, merge_blocks, s) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

// per-device attributes of the chunk kernel, once
cudaError_t prepare_chunk(int dev, bool fp8) {
  const uint32_t bit = fp8 ? 2u : 1u;
  if (g_chunk_prepared[dev].load() & bit) return cudaSuccess;
  const cudaError_t e = chunk_prepare(fp8);
  if (e == cudaSuccess) g_chunk_prepared[dev].fetch_or(bit);
  return e;
}

}  // namespace
}  // namespace mla

MLA_EXPORT size_t mla_chunk_workspace_size(const mla_chunk_params* p, int32_t num_sms) {
  if (check_chunk_params(p) != MLA_OK) return 0;
  if (num_sms <= 0) {
    int dev;
    if (current_device(&dev) != cudaSuccess) return 0;
    num_sms = sm_count(dev);
    if (num_sms <= 0) return 0;
  }
  if (num_sms < 2) return 0;
  return chunk_ws_layout(p->batch, p->num_tokens, p->num_heads, num_sms / 2).total;
}

MLA_EXPORT mla_status mla_chunk_attention(const mla_chunk_params* p, const void* q, const void* kv_cache,
                                          const int32_t* block_table, const int32_t* seq_lens,
                                          const int32_t* cu_q_lens, float softmax_scale, const float* kv_scale,
                                          void* out, float* lse, void* workspace, size_t workspace_bytes,
                                          mla_stream_t stream) {
  const mla_status st = check_chunk_params(p);
  if (st != MLA_OK) return st;
  const bool fp8 = p->kv_dtype == MLA_KV_FP8_E4M3;
  const bool any = p->num_tokens > 0;
  if (!kv_cache || !block_table || !seq_lens || !cu_q_lens || !workspace || (any && (!q || !out || !lse)))
    return MLA_ERR_INVALID_ARG;
  if (fp8 && !kv_scale) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_q_lens, 4) || !aligned(workspace, 256) || !aligned(kv_scale, 4))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || softmax_scale > 3.0e38f || softmax_scale < -3.0e38f)
    return MLA_ERR_INVALID_ARG;
  int dev;
  if (current_device(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  const int nsm = sm_count(dev);
  if (nsm <= 0) return MLA_ERR_CUDA;
  const int pairs = nsm / 2;
  if (pairs < 1) return MLA_ERR_UNSUPPORTED;
  const ChunkWs w = chunk_ws_layout(p->batch, p->num_tokens, p->num_heads, pairs);
  if (workspace_bytes < w.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!get_encoder()) return MLA_ERR_CUDA;
  if (prepare_chunk(dev, fp8) != cudaSuccess) return MLA_ERR_CUDA;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t cap = (int64_t)p->max_blocks_per_seq * p->page_size;
  ChunkSchedArgs sa = chunk_sched_args(ws, w, p->num_heads, p->num_tokens, pairs, fp8);
  sa.seq_lens = seq_lens;
  sa.cu_q = cu_q_lens;
  sa.B = p->batch;
  sa.causal = p->causal;
  sa.max_len = (int)std::min<int64_t>(cap, p->max_seq_len);
  ChunkArgs ca;
  std::memset(&ca, 0, sizeof(ca));
  if (any && !encode_chunk_maps(&ca, q, p->num_tokens, p->num_heads, kv_cache, p->num_pages, p->page_size, fp8))
    return MLA_ERR_INVALID_ARG;
  if (launch_chunk_schedule(sa, s) != cudaSuccess) return MLA_ERR_CUDA;
  if (!any) return MLA_OK;
  ca.block_table = block_table;
  ca.MB = p->max_blocks_per_seq;
  ca.causal = p->causal;
  ChunkCombineArgs cc{};
  cc.block_table = block_table;
  cc.seq_lens = seq_lens;
  cc.cu_q = cu_q_lens;
  cc.B = p->batch;
  cc.MB = p->max_blocks_per_seq;
  cc.P = p->page_size;
  cc.num_pages = p->num_pages;
  cc.max_len = sa.max_len;
  return launch_chunk_pair(ca, cc, sa, ws, w, softmax_scale, kv_scale, out, lse, fp8, pairs, 8 * nsm, s);
}

// ------------------------------------------------------------ rotating append, state merge
MLA_EXPORT mla_status mla_rope_cache_write(const void* latent, int64_t latent_stride, const void* rope,
                                           int64_t rope_stride, const int64_t* positions, const float* cos_sin,
                                           int32_t max_pos, int32_t interleaved, const int64_t* slot_mapping,
                                           int32_t num_tokens, void* kv_cache, int32_t num_pages, int32_t page_size,
                                           int32_t kv_dtype, const float* kv_scale, const void* q_rope,
                                           int64_t q_token_stride, int64_t q_head_stride, int32_t num_heads, void* q,
                                           uint32_t* device_error, mla_stream_t stream) {
  if (num_tokens < 0 || num_pages < 1 || page_size < 1 || max_pos < 1) return MLA_ERR_INVALID_ARG;
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return MLA_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == MLA_KV_FP8_E4M3;
  if ((q_rope == nullptr) != (q == nullptr)) return MLA_ERR_INVALID_ARG;
  if (q != nullptr && num_heads < 1) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (!latent || !rope || !positions || !cos_sin || !slot_mapping || !kv_cache || (fp8 && !kv_scale))
    return MLA_ERR_INVALID_ARG;
  if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(kv_cache, 16) || !aligned(cos_sin, 16) ||
      !aligned(positions, 8) || !aligned(slot_mapping, 8) || !aligned(q, 16) || !aligned(q_rope, 16) ||
      !aligned(kv_scale, 4) || !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  if (latent_stride < kDV || rope_stride < kDRope || latent_stride % 8 != 0 || rope_stride % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  if (q != nullptr && (q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || q_token_stride < 0 || q_head_stride < 0))
    return MLA_ERR_INVALID_ARG;
  if (q != nullptr && num_heads > kMaxRows) return MLA_ERR_UNSUPPORTED;
  // one warp per task, eight to a block: within the grid's limit
  if ((int64_t)num_tokens * (1 + (q != nullptr ? (num_heads + 31) / 32 : 0)) > (int64_t)1 << 33) return MLA_ERR_UNSUPPORTED;
  RopeWriteArgs a{};
  a.latent = static_cast<const __nv_bfloat16*>(latent);
  a.rope = static_cast<const __nv_bfloat16*>(rope);
  a.positions = positions;
  a.slots = slot_mapping;
  a.cos_sin = cos_sin;
  a.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  a.q = static_cast<__nv_bfloat16*>(q);
  a.cache = static_cast<uint8_t*>(kv_cache);
  a.kv_scale = kv_scale;
  a.err = device_error;
  a.latent_stride = latent_stride;
  a.rope_stride = rope_stride;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.total_slots = (int64_t)num_pages * page_size;
  a.n = num_tokens;
  a.H = num_heads;
  a.max_pos = max_pos;
  a.interleaved = interleaved;
  if (launch_rope_write(a, fp8, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

MLA_EXPORT mla_status mla_merge_states(const void* out_a, const float* lse_a, const void* out_b, const float* lse_b,
                                       int64_t num_rows, void* out, float* lse, mla_stream_t stream) {
  if (num_rows < 0) return MLA_ERR_INVALID_ARG;
  if (num_rows == 0) return MLA_OK;
  if (!out_a || !lse_a || !out_b || !lse_b || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (!aligned(out_a, 16) || !aligned(out_b, 16) || !aligned(out, 16) || !aligned(lse_a, 4) || !aligned(lse_b, 4) ||
      !aligned(lse, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_rows > (int64_t)1 << 33) return MLA_ERR_UNSUPPORTED;
  if (launch_merge_states(out_a, lse_a, out_b, lse_b, num_rows, out, lse, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

// -------------------------------------------------------------------- block-sparse attention
MLA_EXPORT mla_status mla_index_cache_write(const void* keys, int64_t key_stride, const int64_t* positions,
                                            const float* cos_sin, int32_t max_pos, int32_t interleaved,
                                            const int64_t* slot_mapping, int32_t num_tokens, void* index_cache,
                                            float* index_scale, int32_t num_pages, int32_t page_size,
                                            const void* queries, int64_t q_token_stride, int64_t q_head_stride,
                                            const float* weights, int32_t num_heads, void* q_index, float* q_weights,
                                            uint32_t* device_error, mla_stream_t stream) {
  if (num_tokens < 0 || num_pages < 1 || page_size < 1 || max_pos < 1) return MLA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return MLA_ERR_INVALID_ARG;
  const bool any = queries != nullptr;
  if (any != (weights != nullptr) || any != (q_index != nullptr) || any != (q_weights != nullptr)) return MLA_ERR_INVALID_ARG;
  if (any && num_heads < 1) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (!keys || !positions || !cos_sin || !slot_mapping || !index_cache || !index_scale) return MLA_ERR_INVALID_ARG;
  if (!aligned(keys, 16) || !aligned(index_cache, 16) || !aligned(index_scale, 4) || !aligned(cos_sin, 16) ||
      !aligned(positions, 8) || !aligned(slot_mapping, 8) || !aligned(queries, 16) || !aligned(q_index, 16) ||
      !aligned(weights, 4) || !aligned(q_weights, 4) || !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  if (key_stride < kDIndex || key_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (any && (q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || q_token_stride < 0 || q_head_stride < 0))
    return MLA_ERR_INVALID_ARG;
  if (any && num_heads > kMaxIndexHeads) return MLA_ERR_UNSUPPORTED;
  IndexWriteArgs a{};
  a.keys = static_cast<const __nv_bfloat16*>(keys);
  a.positions = positions;
  a.slots = slot_mapping;
  a.cos_sin = cos_sin;
  a.queries = static_cast<const __nv_bfloat16*>(queries);
  a.weights = weights;
  a.cache = static_cast<uint8_t*>(index_cache);
  a.scale = index_scale;
  a.q_index = static_cast<uint8_t*>(q_index);
  a.q_weights = q_weights;
  a.err = device_error;
  a.key_stride = key_stride;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.total_slots = (int64_t)num_pages * page_size;
  a.n = num_tokens;
  a.H = num_heads;
  a.max_pos = max_pos;
  a.interleaved = interleaved;
  if (launch_index_write(a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

namespace mla {
namespace {

// what the block-sparse calls share: a ragged batch over pages that hold whole blocks
mla_status check_blocks(const mla_index_params* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_tokens < 0 || p->num_heads < 1 || p->page_size < 1 || p->num_pages < 1 ||
      p->max_blocks_per_seq < 1 || p->max_seq_len < 1 || p->block_size < 1)
    return MLA_ERR_INVALID_ARG;
  if (p->causal != 0 && p->causal != 1) return MLA_ERR_INVALID_ARG;
  if (p->page_size % 8 != 0 || p->page_size > 1024) return MLA_ERR_UNSUPPORTED;
  if (p->block_size % 8 != 0 || p->page_size % p->block_size != 0) return MLA_ERR_UNSUPPORTED;
  if (p->batch > kMaxBatch || p->max_seq_len > kMaxSeqLen || p->num_tokens > kMaxSparseTokens) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->num_pages * p->page_size >= (int64_t)1 << 31) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}
std::atomic<uint32_t> g_index_prepared[kMaxDevices];   // bit 0: index scores, 1: sparse plan

// per-device attributes, once
template <class Prepare>
bool prepare_once(int dev, uint32_t bit, Prepare&& prepare) {
  if (g_index_prepared[dev].load() & bit) return true;
  if (prepare() != cudaSuccess) return false;
  g_index_prepared[dev].fetch_or(bit);
  return true;
}
int blocks_of(int len, int block) { return (len + block - 1) / block; }
// rows of 128 bytes; planes > 0: as many planes of them
bool encode_index_map(CUtensorMap* m, const void* base, int64_t rows, uint32_t box_rows, int64_t planes, uint32_t box_planes) {
  const cuuint64_t dims[3] = {(cuuint64_t)kDIndex, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)kDIndex, (cuuint64_t)kDIndex * (cuuint64_t)rows};
  const cuuint32_t box[3] = {(cuuint32_t)kDIndex, box_rows, box_planes};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, planes > 0 ? 3 : 2, base, dims, strides, box);
}

}  // namespace
}  // namespace mla

MLA_EXPORT mla_status mla_index_scores(const mla_index_params* p, const void* q_index, const float* q_weights,
                                       const void* index_cache, const float* index_scale, const int32_t* block_table,
                                       const int32_t* seq_lens, const int32_t* cu_q_lens, float* scores,
                                       uint32_t* device_error, mla_stream_t stream) {
  const mla_status st = check_blocks(p);
  if (st != MLA_OK) return st;
  if (p->num_heads > kMaxIndexHeads) return MLA_ERR_UNSUPPORTED;
  if (p->num_tokens == 0) return MLA_OK;
  if (!q_index || !q_weights || !index_cache || !index_scale || !block_table || !seq_lens || !cu_q_lens || !scores)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(q_index, 16) || !aligned(q_weights, 4) || !aligned(index_cache, 16) || !aligned(index_scale, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q_lens, 4) || !aligned(scores, 4) ||
      !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  int dev;
  if (current_device(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  const int nsm = sm_count(dev);
  if (nsm <= 0 || !get_encoder() || !prepare_once(dev, 1u, index_scores_prepare)) return MLA_ERR_CUDA;
  IndexScoreArgs a;
  std::memset(&a, 0, sizeof(a));
  const int64_t rows = (int64_t)p->num_pages * p->page_size;
  a.box_rows = box_rows_of(p->page_size, 128);
  a.total_rows = (int32_t)rows;
  int columns, tokens;
  index_scores_group(p->num_tokens, p->batch, p->num_heads, &columns, &tokens);
  if (!encode_index_map(&a.tm_q, q_index, p->num_heads, (uint32_t)columns, p->num_tokens, (uint32_t)tokens) ||
      !encode_index_map(&a.tm_k, index_cache, rows, (uint32_t)a.box_rows, 0, 1))
    return MLA_ERR_INVALID_ARG;
  a.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  a.test_stall = g_test_stall.load(std::memory_order_relaxed);
  a.w = q_weights;
  a.scale = index_scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q_lens;
  a.out = scores;
  a.err = device_error;
  a.B = p->batch;
  a.T = p->num_tokens;
  a.H = p->num_heads;
  a.P = p->page_size;
  a.MB = p->max_blocks_per_seq;
  a.num_pages = p->num_pages;
  a.max_len = (int)std::min<int64_t>((int64_t)p->max_blocks_per_seq * p->page_size, p->max_seq_len);
  a.block = p->block_size;
  a.C = blocks_of(p->max_seq_len, p->block_size);
  a.causal = p->causal;
  if (launch_index_scores(a, nsm, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

MLA_EXPORT mla_status mla_select_blocks(const float* scores, int64_t scores_stride, int32_t num_tokens, int32_t num_blocks,
                                        const int32_t* seq_lens, const int32_t* cu_q_lens, int32_t batch,
                                        int32_t block_size, int32_t top_k, int32_t keep_first, int32_t keep_last,
                                        int32_t causal, int32_t* selected, uint32_t* device_error, mla_stream_t stream) {
  if (num_tokens < 0 || num_blocks < 1 || batch < 1 || block_size < 1 || top_k < 1 || keep_first < 0 || keep_last < 0)
    return MLA_ERR_INVALID_ARG;
  if ((int64_t)keep_first + keep_last > top_k || scores_stride < num_blocks) return MLA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MLA_ERR_INVALID_ARG;
  if (batch > kMaxBatch || num_tokens > kMaxSparseTokens || num_blocks > kMaxSeqLen || top_k > kMaxSeqLen ||
      block_size > kMaxSeqLen)
    return MLA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MLA_OK;
  if (!scores || !seq_lens || !cu_q_lens || !selected) return MLA_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(seq_lens, 4) || !aligned(cu_q_lens, 4) || !aligned(selected, 4) ||
      !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  SelectArgs a{};
  a.scores = scores;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q_lens;
  a.out = selected;
  a.err = device_error;
  a.stride = scores_stride;
  a.B = batch;
  a.T = num_tokens;
  a.C = num_blocks;
  a.K = top_k;
  a.block = block_size;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.causal = causal;
  if (launch_select_blocks(a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

namespace mla {
namespace {

mla_status check_sparse_params(const mla_sparse_params* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  const mla_index_params ip{p->batch, p->num_tokens, p->num_heads, p->page_size, p->num_pages, p->max_blocks_per_seq,
                            p->max_seq_len, p->block_size, p->causal};
  const mla_status st = check_blocks(&ip);
  if (st != MLA_OK) return st;
  if (p->top_k < 1) return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (p->num_heads > kMaxRows || p->top_k > kMaxSeqLen) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)p->num_tokens * p->num_heads > kMaxChunkRows) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}
cudaError_t prepare_decode16(int dev) {
  const uint32_t bit = 1u << variant_bit(16, true);
  if (g_prepared[dev].load() & bit) return cudaSuccess;
  const cudaError_t e = decode_prepare(16, true);
  if (e == cudaSuccess) g_prepared[dev].fetch_or(bit);
  return e;
}

// blocks of the merge: four warps to a row of the most blocks that can be cut, one per worker
int merge_blocks(int64_t blocks, int rows, int workers, int nsm) {
  return (int)std::min<int64_t>(8 * nsm, std::min<int64_t>(blocks, workers) * rows / 2);
}

// the plan, the decode kernel over the tokens' selected blocks, and the merge of cut ones (E4M3, up to 16 rows)
mla_status sparse_few(const mla_sparse_params* p, const SparsePlanArgs& pa, const void* q, const void* kv_cache,
                      float softmax_scale, const float* kv_scale, void* out, float* lse, uint8_t* ws, const SparseWs& w,
                      int nsm, cudaStream_t s) {
  const int rc = 16, H = p->num_heads, per_page = p->page_size / p->block_size;
  const int64_t rows = (int64_t)p->num_pages * p->page_size;
  DecodeArgs da;
  std::memset(&da, 0, sizeof(da));
  da.box_rows = 64;
  if (p->num_tokens > 0 &&
      (!encode_q_map(&da.tm_q, q, p->num_tokens, H, rc) ||
       !encode_kv_map(&da.tm_k, kv_cache, rows, (uint32_t)decode_key_chunks_per_slot(rc, true), 64, true, true) ||
       !encode_kv_map(&da.tm_v, kv_cache, rows, (uint32_t)decode_value_chunks_per_box(rc, true), 64, true, true)))
    return MLA_ERR_INVALID_ARG;
  if (launch_sparse_plan(pa, s) != cudaSuccess) return MLA_ERR_CUDA;
  if (p->num_tokens == 0) return MLA_OK;
  da.kv_cache = kv_cache;
  da.block_table = pa.table;
  da.batch_info = pa.batch_info;
  da.units = reinterpret_cast<const int4*>(pa.sched.units);
  da.cta_first = pa.sched.cta_first;
  da.hdr = pa.sched.hdr;
  da.out = static_cast<__nv_bfloat16*>(out);
  da.lse = lse;
  da.part_o = reinterpret_cast<float*>(ws + w.decode.po_off);
  da.part_lse = reinterpret_cast<float*>(ws + w.decode.plse_off);
  da.err = pa.sched.hdr;
  da.kv_scale = kv_scale;
  da.s_q = 1;
  da.H = H;
  da.R = H;
  da.P = p->block_size;                    // to the decode kernel a block is a page
  da.MB = pa.width;
  da.num_pages = p->num_pages * per_page;
  da.causal = 0;
  da.softmax_scale = softmax_scale;
  da.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  da.test_stall = g_test_stall.load(std::memory_order_relaxed);
  if (launch_decode(da, rc, true, nsm, s) != cudaSuccess) return MLA_ERR_CUDA;
  ChunkCombineArgs cc{};                   // B = 0: the plan has checked the pages
  cc.hdr = pa.sched.hdr;
  cc.err = pa.sched.hdr;
  cc.split_list = pa.sched.split_list;
  cc.part_o = da.part_o;
  cc.part_lse = da.part_lse;
  cc.out = da.out;
  cc.lse = lse;
  if (launch_chunk_combine(cc, rc, merge_blocks(p->num_tokens, rc, nsm, nsm), s) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

// columns of the table of selected blocks
int sparse_width(const mla_sparse_params* p) { return std::min(p->top_k, blocks_of(p->max_seq_len, p->block_size)); }

}  // namespace
}  // namespace mla

MLA_EXPORT size_t mla_sparse_workspace_size(const mla_sparse_params* p, int32_t num_sms) {
  if (check_sparse_params(p) != MLA_OK) return 0;
  if (num_sms <= 0) {
    int dev;
    if (current_device(&dev) != cudaSuccess) return 0;
    num_sms = sm_count(dev);
    if (num_sms <= 0) return 0;
  }
  if (num_sms < 2) return 0;
  return sparse_ws_layout(p->num_tokens, p->num_heads, p->kv_dtype == MLA_KV_FP8_E4M3, p->block_size, sparse_width(p),
                          num_sms)
      .total;
}

MLA_EXPORT mla_status mla_sparse_attention(const mla_sparse_params* p, const void* q, const void* kv_cache,
                                           const int32_t* block_table, const int32_t* seq_lens,
                                           const int32_t* cu_q_lens, const int32_t* selected, float softmax_scale,
                                           const float* kv_scale, void* out, float* lse, void* workspace,
                                           size_t workspace_bytes, mla_stream_t stream) {
  const mla_status st = check_sparse_params(p);
  if (st != MLA_OK) return st;
  const bool fp8 = p->kv_dtype == MLA_KV_FP8_E4M3;
  const bool any = p->num_tokens > 0;
  if (!kv_cache || !block_table || !seq_lens || !cu_q_lens || !workspace || (any && (!q || !out || !lse || !selected)))
    return MLA_ERR_INVALID_ARG;
  if (fp8 && !kv_scale) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_q_lens, 4) || !aligned(selected, 4) || !aligned(workspace, 256) ||
      !aligned(kv_scale, 4))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || softmax_scale > 3.0e38f || softmax_scale < -3.0e38f)
    return MLA_ERR_INVALID_ARG;
  int dev;
  if (current_device(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  const int nsm = sm_count(dev);
  if (nsm <= 0) return MLA_ERR_CUDA;
  const int pairs = nsm / 2;
  if (pairs < 1) return MLA_ERR_UNSUPPORTED;
  const int width = sparse_width(p);
  const SparseWs w = sparse_ws_layout(p->num_tokens, p->num_heads, fp8, p->block_size, width, nsm);
  if (workspace_bytes < w.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!get_encoder()) return MLA_ERR_CUDA;
  if (!prepare_once(dev, 2u, sparse_plan_prepare)) return MLA_ERR_CUDA;
  if (w.few ? prepare_decode16(dev) != cudaSuccess : prepare_chunk(dev, fp8) != cudaSuccess) return MLA_ERR_CUDA;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int per_page = p->page_size / p->block_size;
  SparsePlanArgs pa{};
  if (w.few) {
    pa.few = 1;
    pa.sched.hdr = reinterpret_cast<uint32_t*>(ws);
    pa.sched.cta_first = reinterpret_cast<int32_t*>(ws + w.decode.cta_off);
    pa.sched.split_list = reinterpret_cast<int4*>(ws + w.decode.split_off);
    pa.sched.units = reinterpret_cast<ChunkUnit*>(ws + w.decode.units_off);
    pa.sched.H = p->num_heads;
    pa.sched.workers = nsm;
    pa.sched.setup = 4;                    // as the decode scheduler's
    pa.batch_info = reinterpret_cast<int4*>(ws + w.decode.batch_off);
    pa.out = static_cast<__nv_bfloat16*>(out);
    pa.lse = lse;
  } else {
    pa.sched = chunk_sched_args(ws, w.chunk, p->num_heads, p->num_tokens, pairs, fp8);
  }
  pa.selected = selected;
  pa.block_table = block_table;
  pa.seq_lens = seq_lens;
  pa.cu_q = cu_q_lens;
  pa.table = reinterpret_cast<int32_t*>(ws + w.table_off);
  pa.lens = reinterpret_cast<int32_t*>(ws + w.lens_off);
  pa.B = p->batch;
  pa.T = p->num_tokens;
  pa.K = p->top_k;
  pa.width = width;
  pa.block = p->block_size;
  pa.P = p->page_size;
  pa.MB = p->max_blocks_per_seq;
  pa.num_pages = p->num_pages;
  pa.max_len = (int)std::min<int64_t>((int64_t)p->max_blocks_per_seq * p->page_size, p->max_seq_len);
  pa.causal = p->causal;
  pa.words = (blocks_of(pa.max_len, p->block_size) + 31) / 32;
  if (w.few) return sparse_few(p, pa, q, kv_cache, softmax_scale, kv_scale, out, lse, ws, w, nsm, s);
  ChunkArgs ca;
  std::memset(&ca, 0, sizeof(ca));
  // to the attention kernel a block is a page, and a token a sequence whose pages are its selected blocks
  if (any && !encode_chunk_maps(&ca, q, p->num_tokens, p->num_heads, kv_cache, p->num_pages * per_page, p->block_size, fp8))
    return MLA_ERR_INVALID_ARG;
  if (launch_sparse_plan(pa, s) != cudaSuccess) return MLA_ERR_CUDA;
  if (!any) return MLA_OK;
  ca.block_table = pa.table;
  ca.MB = width;
  ca.causal = 0;
  ChunkCombineArgs cc{};                   // B = 0: the plan has checked the pages
  const int64_t blocks = (int64_t)p->num_tokens * ((p->num_heads + kChunkRows - 1) / kChunkRows);
  return launch_chunk_pair(ca, cc, pa.sched, ws, w.chunk, softmax_scale, kv_scale, out, lse, fp8, pairs,
                           merge_blocks(blocks, kChunkRows, pairs, nsm), s);
}
