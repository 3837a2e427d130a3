// mla_rope.h — arguments of the rotating cache write and of the state merge.
#pragma once
#include "mla_internal.h"

namespace mla {

constexpr int kDRope = 64;

struct RopeWriteArgs {
  const __nv_bfloat16* latent;     // rows of 512, latent_stride elements apart
  const __nv_bfloat16* rope;       // rows of 64, rope_stride elements apart
  const int64_t* positions;
  const int64_t* slots;
  const float* cos_sin;            // [max_pos][32 cosines | 32 sines]
  const __nv_bfloat16* q_rope;     // 64 values per (token, head) at the two strides
  __nv_bfloat16* q;                // [n, H, 576], columns 512.. written; NULL: no queries
  uint8_t* cache;
  const float* kv_scale;
  uint32_t* err;
  int64_t latent_stride, rope_stride, q_token_stride, q_head_stride, total_slots;
  int32_t n, H, max_pos, interleaved, qtasks;
};
cudaError_t launch_rope_write(RopeWriteArgs a, bool fp8, cudaStream_t s);

cudaError_t launch_merge_states(const void* out_a, const float* lse_a, const void* out_b, const float* lse_b,
                                int64_t rows, void* out, float* lse, cudaStream_t s);

}  // namespace mla
