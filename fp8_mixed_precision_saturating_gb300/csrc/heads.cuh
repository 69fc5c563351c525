// heads.cuh -- heads of queries and keys on their way from the projection: the lanes that hold a head's row, its norm,
// its rotation, and where a token of a batch belongs. Used by qk_rope.cu and kv_append.cu.
//
//   n = x w / sqrt(mean(x^2) + eps)             (or x)
//   (a, b) -> amplitude (a cos - b sin, a sin + b cos) for each of rot_dims / 2 pairs of n
//
// Layout of a row. In the vector kernels LPR lanes hold a row, 8 elements each as two chunks of 4 at o0 and o1, chosen so that both
// members of every pair lie in one lane: HALF takes pairs 4 l .. 4 l + 3 as elements 4 l .. and rot_dims / 2 + 4 l ..,
// INTERLEAVED the 8 elements from 8 l on. No element crosses lanes, and the four angles of a lane serve every head of its
// token. Rows that do not come in such chunks (odd sizes, strides or addresses) take the kernels with single elements: a warp per row,
// lane l holding elements l + 32 i, partners read through shared memory.
//
// Angles. p * turns[i] modulo 2^64 is the angle as a fraction of a turn with nothing lost; its top 32 bits are split into a quarter
// turn and a rest within an eighth of a turn either way, whose sine and cosine are taken in fp32 (rest exact to 2^-33 turns).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace fp8gb {
namespace heads {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int32_t pos) {
  const uint32_t a = static_cast<uint32_t>((turns * static_cast<uint64_t>(static_cast<int64_t>(pos))) >> 32);
  const uint32_t quarter = (a + (1u << 29)) >> 30;
  const float r = static_cast<float>(static_cast<int32_t>(a - (quarter << 30))) * 0x1p-31f;  // half turns
  float s, c;
  sincospif(r, &s, &c);
  const bool odd = quarter & 1u;
  float x = odd ? s : c, y = odd ? c : s;
  if ((quarter + 1u) & 2u) x = -x;
  if (quarter & 2u) y = -y;
  return make_float2(x, y);
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A lane's 8 elements as they are in memory, and as the members u, v of 4 pairs.
template <typename T, bool INTER>
struct Raw;
template <>
struct Raw<bf16, false> {
  uint2 a, b;
  __device__ __forceinline__ void load(const bf16* p, int o0, int o1) {
    a = __ldcs(reinterpret_cast<const uint2*>(p + o0));
    b = __ldcs(reinterpret_cast<const uint2*>(p + o1));
  }
  __device__ __forceinline__ void get(float (&u)[4], float (&v)[4]) const {
    u[0] = lo_of(a.x), u[1] = hi_of(a.x), u[2] = lo_of(a.y), u[3] = hi_of(a.y);
    v[0] = lo_of(b.x), v[1] = hi_of(b.x), v[2] = lo_of(b.y), v[3] = hi_of(b.y);
  }
  static __device__ __forceinline__ void put(bf16* p, int o0, int o1, const float (&u)[4], const float (&v)[4]) {
    __stcs(reinterpret_cast<uint2*>(p + o0), make_uint2(pack(u[0], u[1]), pack(u[2], u[3])));
    __stcs(reinterpret_cast<uint2*>(p + o1), make_uint2(pack(v[0], v[1]), pack(v[2], v[3])));
  }
};
template <>
struct Raw<bf16, true> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p, int o0, int) { a = __ldcs(reinterpret_cast<const uint4*>(p + o0)); }
  __device__ __forceinline__ void get(float (&u)[4], float (&v)[4]) const {
    u[0] = lo_of(a.x), u[1] = lo_of(a.y), u[2] = lo_of(a.z), u[3] = lo_of(a.w);
    v[0] = hi_of(a.x), v[1] = hi_of(a.y), v[2] = hi_of(a.z), v[3] = hi_of(a.w);
  }
  static __device__ __forceinline__ void put(bf16* p, int o0, int, const float (&u)[4], const float (&v)[4]) {
    __stcs(reinterpret_cast<uint4*>(p + o0), make_uint4(pack(u[0], v[0]), pack(u[1], v[1]), pack(u[2], v[2]), pack(u[3], v[3])));
  }
};
template <bool INTER>
struct Raw<float, INTER> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int o0, int o1) {
    a = __ldcs(reinterpret_cast<const float4*>(p + o0));
    b = __ldcs(reinterpret_cast<const float4*>(p + o1));
  }
  __device__ __forceinline__ void get(float (&u)[4], float (&v)[4]) const {
    if constexpr (INTER) {
      u[0] = a.x, u[1] = a.z, u[2] = b.x, u[3] = b.z;
      v[0] = a.y, v[1] = a.w, v[2] = b.y, v[3] = b.w;
    } else {
      u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
      v[0] = b.x, v[1] = b.y, v[2] = b.z, v[3] = b.w;
    }
  }
  static __device__ __forceinline__ void put(float* p, int o0, int o1, const float (&u)[4], const float (&v)[4]) {
    if constexpr (INTER) {
      __stcs(reinterpret_cast<float4*>(p + o0), make_float4(u[0], v[0], u[1], v[1]));
      __stcs(reinterpret_cast<float4*>(p + o1), make_float4(u[2], v[2], u[3], v[3]));
    } else {
      __stcs(reinterpret_cast<float4*>(p + o0), make_float4(u[0], u[1], u[2], u[3]));
      __stcs(reinterpret_cast<float4*>(p + o1), make_float4(v[0], v[1], v[2], v[3]));
    }
  }
};

// The same into a row of fp32 in shared memory (put's stores are for global memory alone).
template <bool INTER>
__device__ __forceinline__ void put_shared(float* p, int o0, int o1, const float (&u)[4], const float (&v)[4]) {
  float4* a = reinterpret_cast<float4*>(p + o0);
  float4* b = reinterpret_cast<float4*>(p + o1);
  *a = INTER ? make_float4(u[0], v[0], u[1], v[1]) : make_float4(u[0], u[1], u[2], u[3]);
  *b = INTER ? make_float4(u[2], v[2], u[3], v[3]) : make_float4(v[0], v[1], v[2], v[3]);
}

// Where a lane's chunks begin, and its four angles (cos 1, sin 0 where nothing turns).
struct Lane {
  int o0, o1, pair;
  bool in;
};

template <bool INTER>
__device__ __forceinline__ Lane lane_of(int l, int dim, int rot) {
  Lane a;
  if (INTER) {
    a.o0 = 8 * l;
    a.o1 = a.o0 + 4;
    a.pair = 4 * l;
  } else if (8 * l < rot) {
    a.o0 = 4 * l;
    a.o1 = rot / 2 + 4 * l;
    a.pair = 4 * l;
  } else {
    a.o0 = 8 * l;
    a.o1 = a.o0 + 4;
    a.pair = rot;  // past every pair
  }
  a.in = 8 * l < dim;
  return a;
}

__device__ __forceinline__ void angles(const Lane& a, const uint64_t* turns, int rot, int32_t pos, float amplitude, float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (2 * (a.pair + i) < rot) {
      const float2 t = cos_sin(__ldg(turns + a.pair + i), pos);
      c[i] = t.x * amplitude;
      s[i] = t.y * amplitude;
    }
  }
}

// The weights of a lane's pairs (ones without).
template <bool INTER>
__device__ __forceinline__ void weights(const Lane& a, const float* w, float (&wu)[4], float (&wv)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) wu[i] = wv[i] = 1.0f;
  if (w == nullptr || !a.in) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wu[i] = __ldg(w + (INTER ? a.o0 + 2 * i : a.o0 + i));
    wv[i] = __ldg(w + (INTER ? a.o0 + 2 * i + 1 : a.o1 + i));
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
  return x;
}

__device__ __forceinline__ float element(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ void set_element(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void set_element(float* p, float v) { *p = v; }

// The sequence that row t of a batch belongs to, and its position there; position -1 where there is none. A
// whole warp searches: 32 of the beginnings at a time.
struct Place {
  int seq;
  int64_t pos;
};

__device__ __forceinline__ Place place_of(int64_t t, const Batch& b, int lane) {
  Place r{-1, -1};
  if (b.seqs <= 0 || static_cast<int64_t>(__ldg(b.q_start)) > t) return r;
  int lo = 0, hi = b.seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t i = lo + static_cast<int64_t>(lane) * step;
    const bool before = i < hi && static_cast<int64_t>(__ldg(b.q_start + i)) <= t;
    const int n = max(1, __popc(__ballot_sync(0xFFFFFFFFu, before)));
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  const int64_t first = max(0, __ldg(b.q_start + lo)), end = __ldg(b.q_start + lo + 1);
  if (t >= end || t < first) return r;
  r.seq = lo;
  r.pos = static_cast<int64_t>(max(0, __ldg(b.kv_len + lo))) - (min(end, b.tokens) - first) + (t - first);
  return r;
}

}  // namespace heads
}  // namespace fp8gb
