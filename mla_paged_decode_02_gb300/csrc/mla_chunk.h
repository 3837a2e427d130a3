// mla_chunk.h — plan, workspace layout and kernel arguments of the ragged chunk attention
// (mla_chunk_attention). Not part of the public ABI.
#pragma once
#include "mla_internal.h"

namespace mla {

constexpr int kChunkRows = 128;           // query rows of a block: 64 on each CTA of a pair
constexpr int kChunkTile = 256;           // keys of a tile
constexpr int64_t kMaxChunkRows = (int64_t)1 << 30;   // num_tokens * num_heads

// A unit of work: tiles [tb, te) of one block of up to 128 query rows of a sequence. The
// rows of a sequence are numbered token-major (row = token * H + head).
struct ChunkUnit {
  int32_t b;         // sequence
  int32_t row0;      // first row of the block in q ([T * H] rows)
  int32_t srow0;     // the same, counted from the sequence's first row
  int32_t tiles;     // tb | te << 16
  int32_t slot;      // partial slot, or -1: the unit covers the block's keys and writes the output
  int32_t len;       // keys of the sequence
  int32_t vis;       // keys the sequence's first new token sees (not clamped); not causal: len
  int32_t nrows;     // rows of the block (1..128)
};
static_assert(sizeof(ChunkUnit) == 32, "two 16-byte loads");

struct ChunkWs {
  size_t gbase_off, cta_off, split_off, units_off, plse_off, po_off, total;
  int64_t max_units;
};

// Workspace: [header 256 B][first block of each sequence int32 x (B + 1)][first unit of each
// worker int32 x (workers + 1)][cut blocks int4 x workers][units][partial lse][partial out].
// header words as in mla_internal.h: 0 error bits, 1 units, 2 cut blocks, 3 positions per worker,
// 4 positions charged per block. Every worker boundary cuts at most one block: at most workers - 1
// cut blocks and 2 (workers - 1) partial slots.
inline ChunkWs chunk_ws_layout(int B, int64_t tokens, int H, int workers) {
  ChunkWs w{};
  w.max_units = tokens * H / kChunkRows + B + workers;
  size_t off = 256;
  w.gbase_off = off;  off = align_up(off + sizeof(int32_t) * ((size_t)B + 1), 256);
  w.cta_off = off;    off = align_up(off + sizeof(int32_t) * ((size_t)workers + 1), 256);
  w.split_off = off;  off = align_up(off + sizeof(int4) * (size_t)workers, 256);
  w.units_off = off;  off = align_up(off + sizeof(ChunkUnit) * (size_t)w.max_units, 256);
  w.plse_off = off;   off = align_up(off + sizeof(float) * 2 * (size_t)workers * kChunkRows, 256);
  w.po_off = off;     off = align_up(off + sizeof(float) * 2 * (size_t)workers * kChunkRows * kDV, 256);
  w.total = off;
  return w;
}

struct ChunkSchedArgs {
  const int32_t* seq_lens;
  const int32_t* cu_q;       // [B + 1]
  uint32_t* hdr;
  int32_t* gbase;
  int32_t* cta_first;
  int4* split_list;          // (first row in q, rows, pieces, first partial slot)
  ChunkUnit* units;
  int32_t B, H, causal, max_len, workers, setup;
  int32_t tokens;
};

struct ChunkArgs {
  CUtensorMap tm_q;          // q as [9 chunks][T*H rows][64]: a box is 64 whole rows
  // bf16: the cache as [9 chunks][rows][64], boxes of one chunk x k_box keys and (pages that
  // are a multiple of 64 rows) four chunks x 32 values, else one chunk x v_box values;
  // E4M3: as [rows][576], boxes of 128 columns x k_box / v_box rows. 128-byte swizzle.
  CUtensorMap tm_k, tm_v;
  const int32_t* block_table;
  const ChunkUnit* units;
  const int32_t* cta_first;
  uint32_t* err;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;
  float* part_lse;
  const float* kv_scale;
  int32_t H, P, MB, num_pages, causal;
  int32_t total_rows;        // num_pages * P: a box that starts here reads zeros
  int32_t k_box, v_box;      // rows of one key / value box
  int32_t out_wide;          // out is 32-byte aligned (else 16): the stores that are made
  float softmax_scale;
  uint64_t wait_limit_ns;
  int32_t test_stall;
};

struct ChunkCombineArgs {
  const uint32_t* hdr;
  uint32_t* err;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int32_t B, MB, P, num_pages, max_len;
  const int4* split_list;
  const float* part_o;
  const float* part_lse;
  __nv_bfloat16* out;
  float* lse;
};

cudaError_t launch_chunk_schedule(const ChunkSchedArgs& a, cudaStream_t s);
cudaError_t launch_chunk(const ChunkArgs& a, bool fp8, int pairs, cudaStream_t s);
cudaError_t chunk_prepare(bool fp8);
cudaError_t launch_chunk_combine(const ChunkCombineArgs& a, int grid, cudaStream_t s);

}  // namespace mla
