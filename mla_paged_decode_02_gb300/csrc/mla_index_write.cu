// mla_index_write.cu — new tokens' index keys into the paged index cache, and their index queries:
// rotated, then quantised to E4M3 with a scale for each row of 128.
//
// A row x (a key, or one head of a query) has its last 64 values turned by the token's angles as in
// the rotating cache write (float32, products rounded apart); then
//   m = max(max|x|, 448 x 2^-126),   scale = m / 448,   code = e4m3(x (448 / m)),
// both quotients IEEE float32. A key's codes and scale go to its slot; a query head's scale is
// multiplied into the head's weight, so that w relu(q.k) needs no further factor. A row with a value
// that is not finite gets a NaN scale. (A division for each value instead of one for the row: 41 us against
// 23 then, for 4096 tokens x 64 heads.)
//
// Memory bound at many tokens (4096 x 64 heads 23.7 us for 103 MB, 4.3 TB/s, and 21.9 where inputs stay in L2; 128 x 64
// heads 3.0 and 1.9 us, latency).
// Bytes: 256 in and 132 out per row. Eight lanes share a row (eight values of the fixed half and eight of
// the turned one each); a warp takes four tokens' keys, or 4 or 16 heads of a token.
#include <cuda_fp8.h>
#include "mla_index.h"
#include "mla_ptx.cuh"
#include "mla_rope.h"
#include "../../include/mla.h"

namespace mla {
namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// both members of a turned pair, every product and sum rounded on its own
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}
__device__ __forceinline__ uint2 pack8(const float* q) {
  uint32_t o[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[2 * k], q[2 * k + 1]), __NV_SATFINITE, __NV_E4M3)
                 << (16 * (k & 1));
  return make_uint2(o[0], o[1]);
}
// the codes of 16 values, first and last eight
__device__ __forceinline__ void quantise16(float* x, float inv, uint2& a, uint2& b) {
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] *= inv;
  a = pack8(x);
  b = pack8(x + 8);
}
// the larger, NaN if either is
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// The row of lane group lane / 8, of which this lane holds eight fixed values (v[0]) and eight to be turned
// (v[1]): x receives them all, turned, and the largest magnitude m as above is returned (NaN if a value of
// the row is not finite). Pairs are neighbours, or their members four lanes apart.
__device__ __forceinline__ float row_max(const uint4* v, bool interleaved, bool second, const float* c, const float* s,
                                         float* x) {
  unpack8(v[0], x);
  unpack8(v[1], x + 8);
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) turn(x[8 + 2 * k], x[9 + 2 * k], c[k], s[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float other = __shfl_xor_sync(0xffffffffu, x[8 + k], 4);
      const float u = __fmul_rn(x[8 + k], c[k]), w = __fmul_rn(other, s[k]);
      x[8 + k] = second ? __fadd_rn(u, w) : __fsub_rn(u, w);
    }
  }
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) m = max_nan(m, fabsf(x[k]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m <= 3.402823466e38f ? fmaxf(m, 448.f * 1.17549435e-38f) : __int_as_float(0x7FC00000);
}

}  // namespace

// kIter: heads of a query task / 4.
template <int kIter>
__global__ void __launch_bounds__(256, 3) index_write_kernel(IndexWriteArgs a) {
  const int lane = threadIdx.x & 31, group = lane >> 3;
  const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t key_tasks = (a.n + 3) / 4;
  const bool is_key = task < key_tasks;
  int64_t t;
  int h0 = 0;
  if (is_key) {
    t = min((int64_t)a.n - 1, task * 4 + group);
  } else {
    if (a.queries == nullptr) return;      // the last block's rest
    t = (task - key_tasks) / a.qtasks;
    if (t >= a.n) return;
    h0 = (int)(task - key_tasks - t * a.qtasks) * 4 * kIter + group;
  }
  griddep_wait();                          // the inputs may be the work before's
  griddep_launch_dependents();
  const int64_t pos = a.positions[t];
  const int u = lane & 7;                              // the lane's 8-value unit of each half
  const bool second = (u & 4) != 0;                    // its values are second members of pairs
  // the rows are on their way while the position, and then the cosines and sines, are read
  uint4 v[kIter][2];
  int64_t slot = -1;
  if (is_key) {
    slot = a.slots[t];
    const uint4* r = reinterpret_cast<const uint4*>(a.keys + t * a.key_stride);
    v[0][0] = r[u];
    v[0][1] = r[8 + u];
  } else {
    const __nv_bfloat16* src = a.queries + t * a.q_token_stride;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int h = min(h0 + 4 * i, a.H - 1);
      const uint4* r = reinterpret_cast<const uint4*>(src + h * a.q_head_stride);
      v[i][0] = r[u];
      v[i][1] = r[8 + u];
    }
  }
  const bool live = pos >= 0 && pos < a.max_pos;       // else a padding token, or one that is reported
  float c[8], s[8];
  // its pairs: 4 u .. (neighbours), or 8 (u mod 4) ..
  const float* cs = a.cos_sin + (live ? pos : 0) * kDRope + (a.interleaved ? 4 * u : 8 * (u & 3));
  *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cs);
  *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(cs + 32);
  if (!a.interleaved) {
    *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(cs + 4);
    *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(cs + 36);
  }
  float x[16];
  uint2 q0, q1;
  if (is_key) {
    const float m = row_max(v[0], a.interleaved, second, c, s, x);
    if (task * 4 + group >= a.n || pos < 0) return;
    if (!live || slot >= a.total_slots) {
      if ((lane & 7) == 0 && a.err != nullptr) atomicOr(a.err, !live ? MLA_DEVERR_POSITION : MLA_DEVERR_SLOT);
      return;
    }
    if (slot < 0) return;
    quantise16(x, __fdiv_rn(448.f, m), q0, q1);
    uint2* dst = reinterpret_cast<uint2*>(a.cache + slot * kDIndex);
    dst[u] = q0;
    dst[8 + u] = q1;
    if ((lane & 7) == 0) a.scale[slot] = __fdiv_rn(m, 448.f);
    return;
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int h = h0 + 4 * i;
    const float m = row_max(v[i], a.interleaved, second, c, s, x);
    if (h >= a.H) continue;
    quantise16(x, __fdiv_rn(448.f, m), q0, q1);
    const int64_t row = t * a.H + h;
    uint2* dst = reinterpret_cast<uint2*>(a.q_index + row * kDIndex);
    dst[u] = q0;
    dst[8 + u] = q1;
    if ((lane & 7) == 0) a.q_weights[row] = a.weights[row] * __fdiv_rn(m, 448.f);
  }
}

cudaError_t launch_index_write(IndexWriteArgs a, cudaStream_t s) {
  // 16 heads to a warp (8: 22.5 us against 21.7 for 4096 tokens x 64 heads; 4: 30), 4 where that would leave warps without work
  const bool few = (int64_t)a.n * a.H <= 1 << 15;
  const int per = few ? 4 : 16;
  a.qtasks = a.queries != nullptr ? (a.H + per - 1) / per : 0;
  const int64_t tasks = ((int64_t)a.n + 3) / 4 + (int64_t)a.n * a.qtasks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tasks + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, index_write_kernel<1>, a) : cudaLaunchKernelEx(&cfg, index_write_kernel<4>, a);
}

}  // namespace mla
