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

// Two fp32 values in one 64-bit register: the arithmetic below works on both at once.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ Pair both(float x) { return pair(x, x); }
__device__ __forceinline__ float2 split(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(Pair p) {
  const float2 t = split(p);
  return t.x + t.y;
}
__device__ __forceinline__ Pair pair_of(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t pack2(Pair p) {
  const float2 t = split(p);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(t.y), "f"(t.x));
  return r;
}

// How a row lies in its warps' registers: a warp holds 32 E consecutive columns, a lane E of them. VEC 4: items of 4
// consecutive columns, item i of a lane 128 i columns after its first; VEC 1: element e 32 e columns after it. Either
// way a warp's access is contiguous and an item's place a constant offset. `left`: columns from the lane's first one
// to the row's end; what lies past it reads as zero and is not written. FULL: nothing lies past it (whole warps), so
// nothing is checked.
template <int VEC, int E, bool FULL>
struct Row {
  static __device__ __forceinline__ bool in(int at, int left) { return FULL || at < left; }
  static_assert(E % 4 == 0 && (VEC == 1 || VEC == 4), "items");
  static __device__ __forceinline__ int first(int warp, int lane) { return warp * 32 * E + lane * VEC; }

  // what lies past the row becomes zero
  static __device__ __forceinline__ void clear(Pair (&x)[E / 2], int left) {
    if constexpr (!FULL) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        if constexpr (VEC == 4) {
          if (64 * (i & ~1) >= left) x[i] = both(0.0f);
        } else {
          const float2 v = split(x[i]);
          x[i] = pair(64 * i < left ? v.x : 0.0f, 64 * i + 32 < left ? v.y : 0.0f);
        }
      }
    }
  }

  // stream: rows, read once (kept out of L1); otherwise parameters, which every row reads
  template <bool STREAM>
  static __device__ __forceinline__ void load(const float* p, int left, Pair (&x)[E / 2]) {
    if constexpr (VEC == 4) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4* at = reinterpret_cast<const float4*>(p + 128 * i);
        if (in(128 * i, left)) t = STREAM ? __ldcs(at) : __ldg(at);
        x[2 * i] = pair(t.x, t.y);
        x[2 * i + 1] = pair(t.z, t.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        float lo = 0.0f, hi = 0.0f;
        if (in(64 * e, left)) lo = STREAM ? __ldcs(p + 64 * e) : __ldg(p + 64 * e);
        if (in(64 * e + 32, left)) hi = STREAM ? __ldcs(p + 64 * e + 32) : __ldg(p + 64 * e + 32);
        x[e] = pair(lo, hi);
      }
    }
  }
  template <bool STREAM>
  static __device__ __forceinline__ void load(const bf16* p, int left, Pair (&x)[E / 2]) {
    if constexpr (VEC == 4) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        uint2 t = make_uint2(0u, 0u);
        const uint2* at = reinterpret_cast<const uint2*>(p + 128 * i);
        if (in(128 * i, left)) t = STREAM ? __ldcs(at) : __ldg(at);
        x[2 * i] = pair_of(t.x);
        x[2 * i + 1] = pair_of(t.y);
      }
    } else {
      auto one = [&](int at) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + at;
        uint32_t v = 0;
        if (in(at, left)) v = STREAM ? __ldcs(q) : __ldg(q);
        return __uint_as_float(v << 16);
      };
#pragma unroll
      for (int e = 0; e < E / 2; ++e) x[e] = pair(one(64 * e), one(64 * e + 32));
    }
  }
  // fp32 parameters that a CTA keeps in shared memory; fp32_at: the lane's first column's address
  static __device__ __forceinline__ void load_shared(uint32_t fp32_at, int left, Pair (&x)[E / 2]) {
    static_assert(VEC == 4, "rows of whole 16 bytes");
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (in(128 * i, left)) asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(t.x), "=f"(t.y), "=f"(t.z), "=f"(t.w) : "r"(fp32_at + 512 * i));
      x[2 * i] = pair(t.x, t.y);
      x[2 * i + 1] = pair(t.z, t.w);
    }
  }
  static __device__ __forceinline__ void store(float* p, int left, const Pair (&x)[E / 2]) {
#pragma unroll
    for (int e = 0; e < E / 2; e += VEC == 4 ? 2 : 1) {
      const float2 a = split(x[e]);
      if constexpr (VEC == 4) {
        const float2 b = split(x[e + 1]);
        if (in(64 * e, left)) __stcs(reinterpret_cast<float4*>(p + 64 * e), make_float4(a.x, a.y, b.x, b.y));
      } else {
        if (in(64 * e, left)) __stcs(p + 64 * e, a.x);
        if (in(64 * e + 32, left)) __stcs(p + 64 * e + 32, a.y);
      }
    }
  }
  static __device__ __forceinline__ void store(bf16* p, int left, const Pair (&x)[E / 2]) {
#pragma unroll
    for (int e = 0; e < E / 2; e += VEC == 4 ? 2 : 1) {
      if constexpr (VEC == 4) {
        if (in(64 * e, left)) __stcs(reinterpret_cast<uint2*>(p + 64 * e), make_uint2(pack2(x[e]), pack2(x[e + 1])));
      } else {
        const uint32_t w = pack2(x[e]);
        if (in(64 * e, left)) reinterpret_cast<uint16_t*>(p)[64 * e] = static_cast<uint16_t>(w);
        if (in(64 * e + 32, left)) reinterpret_cast<uint16_t*>(p)[64 * e + 32] = static_cast<uint16_t>(w >> 16);
      }
    }
  }
};

constexpr int kMaxStages = 4;            // rows that a ring in shared memory holds
constexpr int kRingBytes = 216 * 1024;   // of an SM's shared memory for its CTAs' rings

// A row's columns from its copy in shared memory, items of 4 as Row<4, E, FULL> has them.
template <int E, bool FULL, typename T>
__device__ __forceinline__ void held_row(const uint8_t* row, int c, int left, Pair (&x)[E / 2]) {
  const T* p = reinterpret_cast<const T*>(row) + c;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const bool in = FULL || 128 * i < left;
    if constexpr (sizeof(T) == 4) {
      float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (in) q = *reinterpret_cast<const float4*>(p + 128 * i);
      x[2 * i] = pair(q.x, q.y);
      x[2 * i + 1] = pair(q.z, q.w);
    } else {
      uint2 q = make_uint2(0u, 0u);
      if (in) q = *reinterpret_cast<const uint2*>(p + 128 * i);
      x[2 * i] = pair_of(q.x);
      x[2 * i + 1] = pair_of(q.y);
    }
  }
}

// Sums over the warps of a CTA (up to 16), in a fixed order, the same bits on every thread. v: two halves that
// consecutive sums take in turn, so one barrier each is enough: who writes a half again has passed the barrier after
// everyone's read of it. Places of warps that are not there hold zero (clear), so a sum reads all sixteen without a
// loop. A CTA of one warp needs neither.
struct Red {
  __align__(16) float v[2][2][16];
  __device__ __forceinline__ void clear() {  // before the first sum's barrier, by the first 64 threads or fewer
    for (int i = threadIdx.x; i < 64; i += blockDim.x)
      if ((i & 15) >= static_cast<int>(blockDim.x >> 5)) v[0][0][i] = 0.0f;
  }
};
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}
__device__ __forceinline__ float red_sum(const float* r) {
  const float4* q = reinterpret_cast<const float4*>(r);
  Pair a = both(0.0f), b = both(0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = q[i];
    a = add2(a, pair(t.x, t.y));
    b = add2(b, pair(t.z, t.w));
  }
  return sum2(add2(a, b));
}
__device__ __forceinline__ float cta_sum(float s, Red& red, int& turn) {
  s = warp_sum(s);
  if (blockDim.x == 32) return s;
  float* r = red.v[turn][0];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
  __syncthreads();
  return red_sum(r);
}
__device__ __forceinline__ float2 cta_sum(float2 s, Red& red, int& turn) {
  s.x = warp_sum(s.x);
  s.y = warp_sum(s.y);
  if (blockDim.x == 32) return s;
  float *rx = red.v[turn][0], *ry = red.v[turn][1];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) {
    rx[threadIdx.x >> 5] = s.x;
    ry[threadIdx.x >> 5] = s.y;
  }
  __syncthreads();
  return make_float2(red_sum(rx), red_sum(ry));
}

// The same for a team of threads (threadIdx.y) of 2 to WARPS warps that has its own row and its own Red.
template <int WARPS>
__device__ __forceinline__ float team_red(const float* r) {
  const float4* q = reinterpret_cast<const float4*>(r);
  Pair a = both(0.0f), b = both(0.0f);
#pragma unroll
  for (int i = 0; i < WARPS / 4; ++i) {
    const float4 t = q[i];
    a = add2(a, pair(t.x, t.y));
    b = add2(b, pair(t.z, t.w));
  }
  return sum2(add2(a, b));
}
__device__ __forceinline__ void team_sync() { asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory"); }
template <int WARPS>
__device__ __forceinline__ float team_sum(float s, Red& red, int& turn) {
  s = warp_sum(s);
  float* r = red.v[turn][0];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
  team_sync();
  return team_red<WARPS>(r);
}
template <int WARPS>
__device__ __forceinline__ float2 team_sum(float2 s, Red& red, int& turn) {
  s.x = warp_sum(s.x);
  s.y = warp_sum(s.y);
  float *rx = red.v[turn][0], *ry = red.v[turn][1];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) {
    rx[threadIdx.x >> 5] = s.x;
    ry[threadIdx.x >> 5] = s.y;
  }
  team_sync();
  return make_float2(team_red<WARPS>(rx), team_red<WARPS>(ry));
}

// A parameter vector kept in shared memory in fp32, by all threads of a CTA (thread tid of n): p[i] * q[i], `none`
// where there is no p and ones where there is no q. width % 4 == 0.
template <typename T>
__device__ __forceinline__ void keep_product(float* to, const float* p, float none, const T* q, int width, int tid, int n) {
  const bool wide = (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (reinterpret_cast<uintptr_t>(q) & (4 * sizeof(T) - 1)) == 0;
  for (int i = 4 * tid; i < width; i += 4 * n) {
    float a[4] = {none, none, none, none}, b[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    if (wide) {
      if (p != nullptr) {
        const float4 t = __ldg(reinterpret_cast<const float4*>(p + i));
        a[0] = t.x, a[1] = t.y, a[2] = t.z, a[3] = t.w;
      }
      if (q != nullptr) {
        if constexpr (sizeof(T) == 4) {
          const float4 t = __ldg(reinterpret_cast<const float4*>(q + i));
          b[0] = t.x, b[1] = t.y, b[2] = t.z, b[3] = t.w;
        } else {
          const uint2 t = __ldg(reinterpret_cast<const uint2*>(q + i));
          const float2 u = split(pair_of(t.x)), v = split(pair_of(t.y));
          b[0] = u.x, b[1] = u.y, b[2] = v.x, b[3] = v.y;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p != nullptr) a[j] = p[i + j];
        if (q != nullptr) b[j] = load(q + i + j);
      }
    }
    *reinterpret_cast<float4*>(to + i) = make_float4(a[0] * b[0], a[1] * b[1], a[2] * b[2], a[3] * b[3]);
  }
}

// 1 / sqrt(a): the approximation of the special function unit and one Newton step, within 2 units in the last place
// (a division and a square root take some forty instructions of every warp of a row)
__device__ __forceinline__ float inv_sqrt(float a) {
  const float y = rsqrtf(a);
  const float e = fmaf(-a * y, y, 1.0f);  // 1 - a y^2
  return a > 0.0f && a < 3.402823466e38f ? fmaf(0.5f * y, e, y) : y;
}

__device__ __forceinline__ float affine(float z, const float* w, const float* b, int64_t c) {
  if (w != nullptr) z *= w[c];
  return b != nullptr ? z + b[c] : z;
}

// Whether a matrix can be read in pieces of `bytes` bytes: its start and, if there are several, its rows.
inline bool rows_aligned(const void* p, int64_t rows, int64_t ld, int64_t size, int bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || (ld * size) % bytes == 0));
}
__host__ __device__ inline int64_t gate_groups(const NormFwd& f) { return (f.tokens + f.gate_rows - 1) / f.gate_rows; }  // rows of a gate

}  // namespace norms
}  // namespace fp8gb
