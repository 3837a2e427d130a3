// mla_rope_write.cu — new tokens into the paged cache with the position rotation applied on the
// way, and the rotated rope part of their queries.
//
// Token t at position p turns every pair (a, b) of its 64 rope values by the angle of the pair,
//   (a, b) -> (a c - b s, b c + a s),   c, s = cos_sin[p][i], cos_sin[p][32 + i],
// pairs being neighbours (2 i, 2 i + 1) or a half apart (i, i + 32), in float32 with separately
// rounded products, so that the result is the one of the same steps done one by one. Its cache
// row is [latent | rotated rope], its queries' columns 512..575 the rotated query rope parts.
// The rotated value is rounded once: to bf16, or through the float32 quotient by kv_scale to
// E4M3 (the E4M3 cache never sees a bf16 rounding of it).
//
// Memory bound: 1.2 KB in and as much (or half) out per token, and 256 bytes per head. A warp
// takes one task: a token's cache row (72 16-byte groups), or 32 heads of its query rope
// parts, where 4 lanes share a head (16 values each) and a lane keeps its 8 cosines and sines
// in registers over the heads. 4096 tokens x 128 heads, E4M3: 26.5 us for 142 MB (5.4 TB/s; 16 or 64
// heads per task, more resident warps and streaming hints change nothing).
#include <cuda_fp8.h>
#include "mla_internal.h"
#include "mla_rope.h"
#include "../../include/mla.h"

namespace mla {
namespace {

constexpr int kHeadsPerTask = 32;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&h);
}
// both members of a turned pair, every product and sum rounded on its own
__device__ __forceinline__ void turn(float a, float b, float c, float s, float* x, float* y) {
  *x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  *y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_f(w[i]);
    f[2 * i + 1] = hi_f(w[i]);
  }
}

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(256) rope_write_kernel(RopeWriteArgs a) {
  const int lane = threadIdx.x & 31;
  const int per = 1 + a.qtasks;
  const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = task / per;
  const int part = (int)(task - t * per);
  if (t >= a.n) return;
  const int64_t pos = a.positions[t];
  // the token's values are on their way while its position, and then the cosines and sines, are read
  if (part == 0) {
    const int64_t slot = a.slots[t];
    const uint4* lat = reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride);
    const uint4 v[2] = {lat[lane], lat[lane + 32]};
    // rope group g = lane (of 8): columns 8 g .. 8 g + 7
    const int g = lane & 7;
    const uint4 vr = reinterpret_cast<const uint4*>(a.rope + t * a.rope_stride)[g];
    if (pos < 0) return;                             // a padding token
    if (pos >= a.max_pos) {
      if (lane == 0 && a.err != nullptr) atomicOr(a.err, MLA_DEVERR_POSITION);
      return;
    }
    if (slot < 0) return;
    if (slot >= a.total_slots) {
      if (lane == 0 && a.err != nullptr) atomicOr(a.err, MLA_DEVERR_SLOT);
      return;
    }
    const float* cs = a.cos_sin + pos * kDRope;
    float f[8];
    unpack8(vr, f);
    if (a.interleaved) {
      const float4 c = *reinterpret_cast<const float4*>(cs + 4 * g);
      const float4 s = *reinterpret_cast<const float4*>(cs + 32 + 4 * g);
      turn(f[0], f[1], c.x, s.x, &f[0], &f[1]);
      turn(f[2], f[3], c.y, s.y, &f[2], &f[3]);
      turn(f[4], f[5], c.z, s.z, &f[4], &f[5]);
      turn(f[6], f[7], c.w, s.w, &f[6], &f[7]);
    } else {
      // the partner half lives 4 lanes away
      const bool up = (g & 4) != 0;
      const float* cp = cs + 8 * (g & 3);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, f[i], 4);
        float x, y;
        turn(up ? other : f[i], up ? f[i] : other, cp[i], cp[32 + i], &x, &y);
        f[i] = up ? y : x;
      }
    }
    if (!FP8) {
      uint4* dst = reinterpret_cast<uint4*>(a.cache + (size_t)slot * kDQK * 2);
      dst[lane] = v[0];
      dst[lane + 32] = v[1];
      if (lane < 8)
        dst[64 + lane] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else {
      const float scale = __ldg(a.kv_scale);
      uint2* dst = reinterpret_cast<uint2*>(a.cache + (size_t)slot * kDQK);
      auto quant = [&](const float* x) {
        uint32_t o[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 q = make_float2(__fdiv_rn(x[2 * k], scale), __fdiv_rn(x[2 * k + 1], scale));
          const uint32_t b = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
          o[k >> 1] = (k & 1) ? o[k >> 1] | (b << 16) : b;
        }
        return make_uint2(o[0], o[1]);
      };
      if (lane < 8) dst[64 + lane] = quant(f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unpack8(v[h], f);
        dst[lane + 32 * h] = quant(f);
      }
    }
    return;
  }
  // query rope parts of heads h0 ..: lane 4 k + p takes pairs 8 p .. 8 p + 7 of head h0 + k + 8 i
  const int p = lane & 3, h0 = (part - 1) * kHeadsPerTask + (lane >> 2);
  // the 16-byte units of the head's 128 bytes that hold those pairs
  const int u0 = a.interleaved ? 2 * p : p, u1 = a.interleaved ? 2 * p + 1 : p + 4;
  const __nv_bfloat16* src = a.q_rope + t * a.q_token_stride;
  __nv_bfloat16* dst = a.q + t * a.H * kDQK + kDV;
  uint4 v[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = h0 + 8 * i;
    if (h < a.H) {
      const uint4* r = reinterpret_cast<const uint4*>(src + h * a.q_head_stride);
      v[i][0] = r[u0];
      v[i][1] = r[u1];
    }
  }
  if (pos < 0 || pos >= a.max_pos) return;           // reported with the cache row
  const float* cs = a.cos_sin + pos * kDRope;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + 8 * p + i);
    *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + 32 + 8 * p + i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = h0 + 8 * i;
    if (h >= a.H) continue;
    float x[16];
    unpack8(v[i][0], x);
    unpack8(v[i][1], x + 8);
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(x[2 * k], x[2 * k + 1], c[k], s[k], &x[2 * k], &x[2 * k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(x[k], x[8 + k], c[k], s[k], &x[k], &x[8 + k]);
    }
    uint4* o = reinterpret_cast<uint4*>(dst + (int64_t)h * kDQK);
    o[u0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    o[u1] = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
  }
}

cudaError_t launch_rope_write(RopeWriteArgs a, bool fp8, cudaStream_t s) {
  a.qtasks = a.q != nullptr ? (a.H + kHeadsPerTask - 1) / kHeadsPerTask : 0;
  const int64_t tasks = (int64_t)a.n * (1 + a.qtasks);
  const unsigned blocks = (unsigned)((tasks + 7) / 8);
  if (fp8) rope_write_kernel<true><<<blocks, 256, 0, s>>>(a);
  else rope_write_kernel<false><<<blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
