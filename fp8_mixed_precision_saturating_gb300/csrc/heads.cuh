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
// turn and a rest x within an eighth of a turn either way (the lower bits are dropped: at most 2^-32 turns, 1.5 10^-9, one way), whose sine and
// cosine are their Taylor series up to x^9 and x^10: what is left out is below 2 10^-9 and 2 10^-10, fp32 rounds at 3 10^-8. The groups of lanes that hold different rows at
// once share a token's angles: each works out its part of the four and they exchange them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "norm.cuh"

namespace fp8gb {
namespace heads {

using bf16 = __nv_bfloat16;
using norms::add2, norms::both, norms::fma2, norms::mul2, norms::pack2, norms::pair, norms::Pair, norms::pair_of, norms::split, norms::sum2;

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int32_t pos) {
  const uint32_t a = static_cast<uint32_t>((turns * static_cast<uint64_t>(static_cast<int64_t>(pos))) >> 32);
  const uint32_t quarter = (a + (1u << 29)) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(a - (quarter << 30))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float q = x * x;
  const float s = fmaf(x * q, fmaf(q, fmaf(q, fmaf(q, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  const float c = fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const bool odd = quarter & 1u;
  float u = odd ? s : c, v = odd ? c : s;
  if ((quarter + 1u) & 2u) u = -u;
  if (quarter & 2u) v = -v;
  return make_float2(u, v);
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A lane's 8 elements as they are in memory, and as the members u, v of 4 pairs, two pairs to a register pair.
template <typename T, bool INTER>
struct Raw;
template <>
struct Raw<bf16, false> {
  uint2 a, b;
  __device__ __forceinline__ void load(const bf16* p, int o0, int o1) {
    a = __ldcs(reinterpret_cast<const uint2*>(p + o0));
    b = __ldcs(reinterpret_cast<const uint2*>(p + o1));
  }
  __device__ __forceinline__ void get(Pair (&u)[2], Pair (&v)[2]) const {
    u[0] = pair_of(a.x), u[1] = pair_of(a.y);
    v[0] = pair_of(b.x), v[1] = pair_of(b.y);
  }
  static __device__ __forceinline__ void put(bf16* p, int o0, int o1, const Pair (&u)[2], const Pair (&v)[2]) {
    __stcs(reinterpret_cast<uint2*>(p + o0), make_uint2(pack2(u[0]), pack2(u[1])));
    __stcs(reinterpret_cast<uint2*>(p + o1), make_uint2(pack2(v[0]), pack2(v[1])));
  }
};
template <>
struct Raw<bf16, true> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p, int o0, int) { a = __ldcs(reinterpret_cast<const uint4*>(p + o0)); }
  __device__ __forceinline__ void get(Pair (&u)[2], Pair (&v)[2]) const {
    u[0] = pair(lo_of(a.x), lo_of(a.y)), u[1] = pair(lo_of(a.z), lo_of(a.w));
    v[0] = pair(hi_of(a.x), hi_of(a.y)), v[1] = pair(hi_of(a.z), hi_of(a.w));
  }
  static __device__ __forceinline__ void put(bf16* p, int o0, int, const Pair (&u)[2], const Pair (&v)[2]) {
    const float2 u0 = split(u[0]), u1 = split(u[1]), v0 = split(v[0]), v1 = split(v[1]);
    __stcs(reinterpret_cast<uint4*>(p + o0), make_uint4(pack(u0.x, v0.x), pack(u0.y, v0.y), pack(u1.x, v1.x), pack(u1.y, v1.y)));
  }
};
template <bool INTER>
struct Raw<float, INTER> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int o0, int o1) {
    a = __ldcs(reinterpret_cast<const float4*>(p + o0));
    b = __ldcs(reinterpret_cast<const float4*>(p + o1));
  }
  __device__ __forceinline__ void get(Pair (&u)[2], Pair (&v)[2]) const {
    if constexpr (INTER) {
      u[0] = pair(a.x, a.z), u[1] = pair(b.x, b.z);
      v[0] = pair(a.y, a.w), v[1] = pair(b.y, b.w);
    } else {
      u[0] = pair(a.x, a.y), u[1] = pair(a.z, a.w);
      v[0] = pair(b.x, b.y), v[1] = pair(b.z, b.w);
    }
  }
  static __device__ __forceinline__ void arrange(const Pair (&u)[2], const Pair (&v)[2], float4& x, float4& y) {
    const float2 u0 = split(u[0]), u1 = split(u[1]), v0 = split(v[0]), v1 = split(v[1]);
    x = INTER ? make_float4(u0.x, v0.x, u0.y, v0.y) : make_float4(u0.x, u0.y, u1.x, u1.y);
    y = INTER ? make_float4(u1.x, v1.x, u1.y, v1.y) : make_float4(v0.x, v0.y, v1.x, v1.y);
  }
  static __device__ __forceinline__ void put(float* p, int o0, int o1, const Pair (&u)[2], const Pair (&v)[2]) {
    float4 x, y;
    arrange(u, v, x, y);
    __stcs(reinterpret_cast<float4*>(p + o0), x);
    __stcs(reinterpret_cast<float4*>(p + o1), y);
  }
};

// The same into a row of fp32 in shared memory (put's stores are for global memory alone).
template <bool INTER>
__device__ __forceinline__ void put_shared(float* p, int o0, int o1, const Pair (&u)[2], const Pair (&v)[2]) {
  float4 x, y;
  Raw<float, INTER>::arrange(u, v, x, y);
  *reinterpret_cast<float4*>(p + o0) = x;
  *reinterpret_cast<float4*>(p + o1) = y;
}

// Where a lane's chunks begin, the first of its four pairs, and how many of them turn.
struct Lane {
  int o0, o1, pair, turned;
  bool in;
};

template <bool INTER>
__device__ __forceinline__ Lane lane_of(int l, int dim, int rot) {
  Lane a;
  if (INTER) {
    a.o0 = 8 * l;
    a.o1 = a.o0 + 4;
    a.pair = 4 * l;
    a.turned = min(max(rot / 2 - a.pair, 0), 4);
  } else if (8 * l < rot) {
    a.o0 = 4 * l;
    a.o1 = rot / 2 + 4 * l;
    a.pair = 4 * l;
    a.turned = 4;
  } else {
    a.o0 = 8 * l;
    a.o1 = a.o0 + 4;
    a.pair = rot;  // past every pair
    a.turned = 0;
  }
  a.in = 8 * l < dim;
  return a;
}

template <int LPR>
__device__ __forceinline__ void angles(const Lane& a, const uint64_t* turns, int rot, int32_t pos, float amplitude, float (&c)[4], float (&s)[4]) {
  constexpr int RPW = 32 / LPR, MINE = 4 / RPW;  // (rows of 8 lanes and more: at most 4 groups)
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  float2 mine[MINE];
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    const int pair = a.pair + j * RPW + sub;
    mine[j] = make_float2(1.0f, 0.0f);
    if (2 * pair < rot) {
      mine[j] = cos_sin(__ldg(turns + pair), pos);
      mine[j].x *= amplitude;
      mine[j].y *= amplitude;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    c[k] = __shfl_sync(0xFFFFFFFFu, mine[k / RPW].x, (k % RPW) * LPR + l);
    s[k] = __shfl_sync(0xFFFFFFFFu, mine[k / RPW].y, (k % RPW) * LPR + l);
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

// What the forward multiplies a pair's members with: y_u = r (u uc + v nvs), y_v = r (u us + v vc), r the row's 1 / root.
struct Factors {
  Pair uc[2], us[2], vc[2], nvs[2];
};
__device__ __forceinline__ Factors factors(const float (&c)[4], const float (&s)[4], const float (&wu)[4], const float (&wv)[4]) {
  Factors f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Pair pc = pair(c[2 * k], c[2 * k + 1]), ps = pair(s[2 * k], s[2 * k + 1]), pu = pair(wu[2 * k], wu[2 * k + 1]), pv = pair(wv[2 * k], wv[2 * k + 1]);
    f.uc[k] = mul2(pu, pc);
    f.us[k] = mul2(pu, ps);
    f.vc[k] = mul2(pv, pc);
    f.nvs[k] = mul2(mul2(pv, ps), both(-1.0f));
  }
  return f;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
  return x;
}

// x's members as a pair's other ones take them: nothing of those that do not turn, whose sine of 0 times an infinity or a NaN would be no 0
// (`nothing`: a zero whose product with the sine is -0, so that a -0 stays one).
// A lane's pairs turn together with HALF. (PARTIAL: kernels of heads that turn in part, so that the others do without the selections. 8192 tokens of 40
// heads of 128 in bf16 with norms, halves and interleaved: forward 29.4 and 28.6 us, half of each head turning 30.5 and 29.3; gradient
// 53.4 and 54.5, 53.9 and 62.1.)
template <bool INTER, bool PARTIAL>
__device__ __forceinline__ void turning(int turned, float nothing, const Pair (&x)[2], Pair (&t)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    t[k] = x[k];
    if constexpr (PARTIAL) {
      const float2 a = split(x[k]);
      t[k] = pair((INTER ? 2 * k < turned : turned > 0) ? a.x : nothing, (INTER ? 2 * k + 1 < turned : turned > 0) ? a.y : nothing);
    }
  }
}

template <int LPR, bool NORM, bool INTER, bool PARTIAL>
__device__ __forceinline__ void turn(const Lane& a, const Factors& f, float inv_dim, float eps, const Pair (&u)[2], const Pair (&v)[2], Pair (&yu)[2], Pair (&yv)[2]) {
  Pair tu[2], tv[2];
  turning<INTER, PARTIAL>(a.turned, -0.0f, u, tu);  // (times us)
  turning<INTER, PARTIAL>(a.turned, 0.0f, v, tv);   // (times nvs)
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    yu[k] = fma2(u[k], f.uc[k], mul2(tv[k], f.nvs[k]));
    yv[k] = fma2(tu[k], f.us[k], mul2(v[k], f.vc[k]));
  }
  if constexpr (NORM) {
    const float q = sum2(fma2(u[0], u[0], fma2(u[1], u[1], fma2(v[0], v[0], mul2(v[1], v[1])))));
    const Pair r = both(rsqrtf(fmaf(row_sum<LPR>(q), inv_dim, eps)));
#pragma unroll
    for (int k = 0; k < 2; ++k) yu[k] = mul2(yu[k], r), yv[k] = mul2(yv[k], r);
  }
}

__device__ __forceinline__ float element(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ void set_element(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void set_element(float* p, float v) { *p = v; }

// The sequence that row t of a batch belongs to, and its position there; sequence and position -1 where there is none. A
// whole warp searches: 32 of the beginnings at a time, as if they rise. A row that is not found so (a row of nobody is not, either) is looked for in
// every sequence, since beginnings may fall, as in the zeros of unused entries.
struct Place {
  int seq;
  int64_t pos;
};

__device__ __forceinline__ bool holds(const Batch& b, int seq, int64_t t) {
  return static_cast<int64_t>(__ldg(b.q_start + seq)) <= t && t < static_cast<int64_t>(__ldg(b.q_start + seq + 1));
}

__device__ __forceinline__ Place place_of(int64_t t, const Batch& b, int lane) {
  Place r{-1, -1};
  if (b.seqs <= 0) return r;
  int lo = 0, hi = b.seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t i = lo + static_cast<int64_t>(lane) * step;
    const bool before = i < hi && static_cast<int64_t>(__ldg(b.q_start + i)) <= t;
    const int n = max(1, __popc(__ballot_sync(0xFFFFFFFFu, before)));
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  if (!holds(b, lo, t)) {
    lo = -1;
#pragma unroll 1
    for (int64_t s = 0; s < b.seqs && lo < 0; s += 256) {  // 8 of a lane's at a time, their loads together (past the end: an empty sequence)
      const int32_t* q = b.q_start + s;
      const int left = static_cast<int>(min(b.seqs - s, int64_t{512})), row = static_cast<int>(t);
      int32_t from[8], to[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) from[j] = __ldg(q + min(32 * j + lane, left)), to[j] = __ldg(q + min(32 * j + lane + 1, left));
      uint32_t at = 256;
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (from[j] <= row && row < to[j]) at = 32 * j + lane;
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      if (at < 256) lo = static_cast<int>(s) + static_cast<int>(at);
    }
    if (lo < 0) return r;
  }
  const int64_t first = max(0, __ldg(b.q_start + lo)), end = __ldg(b.q_start + lo + 1);
  r.seq = lo;
  r.pos = static_cast<int64_t>(max(0, __ldg(b.kv_len + lo))) - (min(end, b.tokens) - first) + (t - first);
  return r;
}

}  // namespace heads
}  // namespace fp8gb
