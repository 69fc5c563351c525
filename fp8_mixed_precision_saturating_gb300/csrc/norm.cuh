// norm.cuh -- what the forward and the backward of the norms around a block share.
//
//   n = norm_post(o) w_post + b_post;  r' = alpha r + gate n;  h = norm_pre(r') w_pre + b_pre
//
// (include/fp8gb.h, "The norms around a block"). Every norm is z = (x - mean) rstd, then z w + b.
// Statistics and sums are held in fp32; a layer norm's variance is taken about its mean (two
// passes over the row), so a large mean does not cancel it away.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace fp8gb {
namespace norms {

constexpr int kNone = 0, kRms = 1, kLayer = 2;
constexpr int kThreads = 256;  // of the kernels that take any width and alignment

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// VEC consecutive elements. stream: data read or written once (kept out of L1, evicted first from
// L2); otherwise parameters, which every row reads.
template <int VEC>
__device__ __forceinline__ void load_stream(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 t = __ldcs(reinterpret_cast<const float4*>(p));
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
    v[0] = __ldcs(p);
  }
}
__device__ __forceinline__ void unpack4(uint2 t, float (&v)[4]) {
  v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xFFFF0000u);
  v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xFFFF0000u);
}
template <int VEC>
__device__ __forceinline__ void load_stream(const bf16* p, float (&v)[VEC]) {
  if constexpr (VEC == 4)
    unpack4(__ldcs(reinterpret_cast<const uint2*>(p)), v);
  else
    v[0] = __uint_as_float(static_cast<uint32_t>(__ldcs(reinterpret_cast<const uint16_t*>(p))) << 16);
}
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 t = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
    v[0] = __ldg(p);
  }
}
template <int VEC>
__device__ __forceinline__ void load_param(const bf16* p, float (&v)[VEC]) {
  if constexpr (VEC == 4)
    unpack4(__ldg(reinterpret_cast<const uint2*>(p)), v);
  else
    v[0] = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p))) << 16);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int VEC>
__device__ __forceinline__ void store_stream(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  else
    __stcs(p, v[0]);
}
template <int VEC>
__device__ __forceinline__ void store_stream(bf16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3])));
  else
    *p = __float2bfloat16_rn(v[0]);
}

// Sums of two values over the warps of a CTA (all of them; `warps` of them), the same bits on every
// thread. red: 2 x 32 values that consecutive sums take in turn, so one barrier each is enough: who
// writes a half again has passed the barrier after everyone's read of it.
__device__ __forceinline__ float2 warp_sum2(float2 s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
    s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
  }
  return s;
}
__device__ __forceinline__ float2 cta_sum2(float2 s, float2 (*red)[32], int& turn, int warps) {
  s = warp_sum2(s);
  if (warps == 1) return s;
  float2* r = red[turn];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
  __syncthreads();
  s = r[0];
  for (int w = 1; w < warps; ++w) {
    s.x += r[w].x;
    s.y += r[w].y;
  }
  return s;
}

__device__ __forceinline__ float affine(float z, const float* w, const float* b, int64_t c) {
  if (w != nullptr) z *= w[c];
  return b != nullptr ? z + b[c] : z;
}

// Whether a matrix can be read in pieces of `bytes` bytes: its start and its rows.
inline bool rows_aligned(const void* p, int64_t ld, int64_t size, int bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * size) % bytes == 0);
}

}  // namespace norms
}  // namespace fp8gb
