// mla_index.h — arguments of the block-sparse operators: index cache write, block scores, block
// selection, and the plan of the sparse attention. Not part of the public ABI.
#pragma once
#include "mla_chunk.h"

namespace mla {

constexpr int kDIndex = 128;              // width of an index key and of an index query head
constexpr int kMaxIndexHeads = 128;
constexpr int kMaxSparseTokens = 1 << 20;

struct IndexWriteArgs {
  const __nv_bfloat16* keys;       // rows of 128, key_stride elements apart
  const int64_t* positions;
  const int64_t* slots;
  const float* cos_sin;            // [max_pos][32 cosines | 32 sines]
  const __nv_bfloat16* queries;    // 128 values per (token, head) at the two strides; NULL: none
  const float* weights;            // [n, H]
  uint8_t* cache;                  // [slots][128] E4M3
  float* scale;                    // [slots]
  uint8_t* q_index;                // [n, H, 128] E4M3
  float* q_weights;                // [n, H]
  uint32_t* err;
  int64_t key_stride, q_token_stride, q_head_stride, total_slots;
  int32_t n, H, max_pos, interleaved, qtasks;
};
cudaError_t launch_index_write(IndexWriteArgs a, cudaStream_t s);

struct IndexScoreArgs {
  CUtensorMap tm_q;                // [T][H][128] E4M3, boxes of a group's tokens (zeros behind the last head)
  CUtensorMap tm_k;                // [num_pages * P rows][128] E4M3, boxes of box_rows rows
  const float* w;                  // [T, H]
  const float* scale;              // [num_pages * P]
  const int32_t* block_table;      // [B, MB]
  const int32_t* seq_lens;
  const int32_t* cu_q;             // [B + 1]
  float* out;                      // [T, C]
  uint32_t* err;
  int32_t B, T, H, P, MB, num_pages, max_len, block, C, causal;
  int32_t box_rows, total_rows;
  int32_t TG, tg_log2;             // tokens of a group, a power of two
  int32_t q_rows, units, key_slots;   // rows of a query buffer, query buffers, tiles of keys in shared memory
  int32_t unit_blocks, usual_blocks;  // blocks of a unit: at most; unless the kernel chooses
  int32_t choose, step_blocks, step_tiles;   // least whole blocks of whole tiles
  float by_grid;                      // 1 / CTAs
  uint32_t block_inv, page_inv;    // 2^32 / block, 2^32 / P, rounded up
  uint32_t by_blocks, by_heads;    // (2^32 - 1) / unit_blocks, / H, rounded down
  int32_t test_stall;
  uint64_t wait_limit_ns;
};
cudaError_t index_scores_prepare();   // per-device kernel attributes
void index_scores_group(int T, int B, int H, int* columns, int* tokens);
cudaError_t launch_index_scores(IndexScoreArgs a, int num_sms, cudaStream_t s);

struct SelectArgs {
  const float* scores;             // rows of C, stride elements apart
  const int32_t* seq_lens;
  const int32_t* cu_q;             // [B + 1]
  int32_t* out;                    // [T, K]
  uint32_t* err;
  int64_t stride;
  int32_t B, T, C, K, block, keep_first, keep_last, causal;
};
cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t s);

// The plan of a sparse attention: each token becomes a sequence of its own whose pages are its
// selected blocks, ascending, for the attention kernels.
struct SparsePlanArgs {
  ChunkSchedArgs sched;            // hdr, cta_first, split_list, units, H, workers, setup
  const int32_t* selected;         // [T, K]
  const int32_t* block_table;      // [B, MB]
  const int32_t* seq_lens;
  const int32_t* cu_q;             // [B + 1]
  int32_t* table;                  // [T, width]: selected blocks in units of `block` rows of the pool
  int32_t* lens;                   // [T]: keys of those blocks that the token sees (for many tokens)
  int32_t B, T, K, width, block, P, MB, num_pages, max_len, causal;
  int32_t words;                   // 32-bit words of a token's set of blocks
  // for the decode kernel: units and cut blocks in its form, lengths, and the results of tokens without keys
  int32_t few;
  int4* batch_info;                // [T]
  __nv_bfloat16* out;
  float* lse;
};
constexpr int kPlanCtas = 8;       // one cluster
cudaError_t sparse_plan_prepare();    // per-device kernel attributes
cudaError_t launch_sparse_plan(const SparsePlanArgs& a, cudaStream_t s);

// Up to 16 rows with the FP8 cache and blocks of whole 64-row boxes go to the decode kernel (16 rows, keys
// on M), everything else to the chunk attention's (128 rows on M). The kernels alone, 16 heads x 2041 keys,
// E4M3: 15.6 us against 17.6 for 16 tokens, 28.6 against 35.8 for 64, 79 against 101 for 256. Calls: blocks of
// 32 rows, 512 tokens, 192 against 183 us; 32 heads, 64 tokens, 49 against 46; bf16, 16 heads, 1 to 4 tokens
// about equal, 16 tokens 25.4 against 28.3, 64 54 against 51, 152 77 against 87, 512 223 against 259: there the decode
// kernel would gain a tenth from some 100 tokens on, which is not made use of.
inline bool sparse_few_rows(int H, bool fp8, int block) { return fp8 && H <= 16 && block % 64 == 0; }

struct SparseWs {
  bool few;
  ChunkWs chunk;                   // of the chunk attention's kernels, or
  WsLayout decode;                 // of the decode kernel's
  size_t lens_off, table_off, total;
};
inline SparseWs sparse_ws_layout(int64_t tokens, int H, bool fp8, int block, int width, int num_sms) {
  SparseWs w{};
  w.few = sparse_few_rows(H, fp8, block);
  size_t off;
  if (w.few) {
    w.decode = ws_layout((int)tokens, make_plan(H, fp8), num_sms);
    off = w.decode.total;
  } else {
    w.chunk = chunk_ws_layout((int)tokens, tokens, H, num_sms / 2);
    off = w.chunk.total;
  }
  w.lens_off = off;   off = align_up(off + sizeof(int32_t) * (size_t)tokens, 256);
  w.table_off = off;  off = align_up(off + sizeof(int32_t) * (size_t)tokens * (size_t)width, 256);
  w.total = off;
  return w;
}

}  // namespace mla
