// mla_index_write.cu — new tokens' index keys into the paged index cache, and their index queries:
// rotated, then quantised to E4M3 with a scale for each row of 128.
//
// A row x (a key, or one head of a query) has its last 64 values turned by the token's angles as in
// the rotating cache write (float32, products rounded apart); then
//   scale = max(max|x| / 448, 2^-126),   code = e4m3(x / scale),
// both quotients IEEE float32. A key's codes and scale go to its slot; a query head's scale is
// multiplied into the head's weight, so that w relu(q.k) needs no further factor. A row with a value
// that is not finite gets a NaN scale.
//
// Memory bound: 256 bytes in and 132 out per row. Eight lanes share a row (16 values each: the first
// four lanes the fixed half, the others eight pairs), a warp takes a token's key or 16 of its heads.
#include <cuda_fp8.h>
#include "mla_index.h"
#include "mla_rope.h"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kHeadsPerTask = 16;

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
__device__ __forceinline__ uint2 quantise8(const float* x, float scale) {
  uint32_t o[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 q = make_float2(__fdiv_rn(x[2 * k], scale), __fdiv_rn(x[2 * k + 1], scale));
    o[k >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (16 * (k & 1));
  }
  return make_uint2(o[0], o[1]);
}

// The row of lane group lane / 8, of which this lane holds two 16-byte units (u0, u1) as v: turned,
// and its scale. x receives the 16 values.
__device__ __forceinline__ float row_scale(const uint4* v, int p, bool turned, bool interleaved, const float* c,
                                           const float* s, float* x) {
  unpack8(v[0], x);
  unpack8(v[1], x + 8);
  if (turned) {
    if (interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(x[2 * k], x[2 * k + 1], c[k], s[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(x[k], x[8 + k], c[k], s[k]);
    }
  }
  float m = 0.f;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    m = fmaxf(m, fabsf(x[k]));
    bad |= !(fabsf(x[k]) <= 3.402823466e38f);
  }
  if (bad) m = INFINITY;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m == INFINITY ? __int_as_float(0x7FC00000) : fmaxf(__fdiv_rn(m, 448.f), 1.17549435e-38f);
}

}  // namespace

__global__ void __launch_bounds__(256) index_write_kernel(IndexWriteArgs a) {
  const int lane = threadIdx.x & 31;
  const int per = 1 + a.qtasks;
  const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = task / per;
  const int part = (int)(task - t * per);
  if (t >= a.n) return;
  const int64_t pos = a.positions[t];
  const int p = lane & 3;
  const bool turned = (lane & 4) != 0;
  // the lane's 8-value units of the row's 16: pairs are neighbours, or 32 columns (4 units) apart
  const bool apart = turned && !a.interleaved;
  const int u0 = (turned ? 8 : 0) + (apart ? p : 2 * p), u1 = apart ? u0 + 4 : u0 + 1;
  // the rows are on their way while the position, and then the cosines and sines, are read
  constexpr int kIter = kHeadsPerTask / 4;
  uint4 v[kIter][2];
  const int h0 = (part - 1) * kHeadsPerTask + (lane >> 3);
  int64_t slot = -1;
  if (part == 0) {
    slot = a.slots[t];
    const uint4* r = reinterpret_cast<const uint4*>(a.keys + t * a.key_stride);
    v[0][0] = r[u0];
    v[0][1] = r[u1];
  } else {
    const __nv_bfloat16* src = a.queries + t * a.q_token_stride;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int h = min(h0 + 4 * i, a.H - 1);
      const uint4* r = reinterpret_cast<const uint4*>(src + h * a.q_head_stride);
      v[i][0] = r[u0];
      v[i][1] = r[u1];
    }
  }
  if (pos < 0) return;                                 // a padding token
  if (pos >= a.max_pos) {
    if (part == 0 && lane == 0 && a.err != nullptr) atomicOr(a.err, MLA_DEVERR_POSITION);
    return;
  }
  float c[8], s[8];
  const float* cs = a.cos_sin + pos * kDRope + 8 * p;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
    *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + 32 + i);
  }
  float x[16];
  if (part == 0) {
    if (slot < 0) return;
    if (slot >= a.total_slots) {
      if (lane == 0 && a.err != nullptr) atomicOr(a.err, MLA_DEVERR_SLOT);
      return;
    }
    const float scale = row_scale(v[0], p, turned, a.interleaved, c, s, x);
    if (lane >= 8) return;                             // the four lane groups hold the same row
    uint2* dst = reinterpret_cast<uint2*>(a.cache + slot * kDIndex);
    dst[u0] = quantise8(x, scale);
    dst[u1] = quantise8(x + 8, scale);
    if (lane == 0) a.scale[slot] = scale;
    return;
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int h = h0 + 4 * i;
    const float scale = row_scale(v[i], p, turned, a.interleaved, c, s, x);
    if (h >= a.H) continue;
    const int64_t row = t * a.H + h;
    uint2* dst = reinterpret_cast<uint2*>(a.q_index + row * kDIndex);
    dst[u0] = quantise8(x, scale);
    dst[u1] = quantise8(x + 8, scale);
    if ((lane & 7) == 0) a.q_weights[row] = a.weights[row] * scale;
  }
}

cudaError_t launch_index_write(IndexWriteArgs a, cudaStream_t s) {
  a.qtasks = a.queries != nullptr ? (a.H + kHeadsPerTask - 1) / kHeadsPerTask : 0;
  const int64_t tasks = (int64_t)a.n * (1 + a.qtasks);
  index_write_kernel<<<(unsigned)((tasks + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
