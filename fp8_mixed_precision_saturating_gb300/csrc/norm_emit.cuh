// norm_emit.cuh -- what the forward kernels of the norms share beyond norm.cuh: h in 4 bits, and the choice of the
// kernel for many rows.
#pragma once
#include "fp4.cuh"
#include "norm.cuh"

namespace fp8gb {

// Many rows of whole 16 bytes with a block's output (norm_fwd_ring.cu); taken: whether it was one for that kernel.
cudaError_t launch_norm_fwd_ring(const NormFwd& f, cudaStream_t stream, bool* taken);

namespace norms {

inline uint32_t gate_rows_of(const NormFwd& f) { return static_cast<uint32_t>(f.gate_rows); }

// The quotients that NVFP4's group factors are made of (fp4::quotient), by 8 threads; the caller puts a barrier before emit_row.
__device__ __forceinline__ float h_scale_of(const NormFwd& f) { return f.h_scale != nullptr ? __ldg(f.h_scale) : 1.0f; }
__device__ __forceinline__ void fill_table(const NormFwd& f, float* table, int tid) {
  if (f.hq != nullptr && f.h_fmt == 0 && tid < 8) table[tid] = fp4::quotient(h_scale_of(f), tid);
}

// NVFP4's scale byte and factor by divisions, out of the way of the kernels' own instructions: inline, its code took 1.5 % of
// the time of kernels that never ran it.
static __device__ __noinline__ uint2 divided(uint32_t a, float s, uint32_t least) {
  float mul;
  const uint32_t c = fp4::group_scale<0>(a, s, least, mul);
  return make_uint2(c, __float_as_uint(mul));
}

// The group's scale byte and the factor of its elements. The caller's tensor scale may be any number: outside
// [2^-100, 2^100] the table's quotients could round where the division does not, so it is divided then (tabled: not).
template <int FMT>
__device__ __forceinline__ uint32_t h_group_scale(uint32_t a, float s, uint32_t least, bool tabled, const float* table, float& mul) {
  if constexpr (FMT == 0) {
    if (tabled) return fp4::group_scale_nv(a, s, 1u, table, mul);
    const uint2 r = divided(a, s, least);
    mul = __uint_as_float(r.y);
    return r.x;
  } else {
    return fp4::group_scale<FMT>(a, s, least, mul);
  }
}

// |a| and |b|'s larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// One element of h a lane as a 4-bit code, its group held by neighbouring lanes. q, sf: the row's codes, and its byte of
// group 0 in the scale atoms.
template <int FMT>
__device__ __forceinline__ void emit_single(float h, int c, int width, float s, uint32_t least, bool tabled, const float* table, uint8_t* q, uint8_t* sf) {
  constexpr int G = fp4::F4<FMT>::kGroup;
  uint32_t a = __float_as_uint(h) & 0x7FFFFFFFu;
  const uint32_t mask = G == 32 ? 0xFFFFFFFFu : 0xFFFFu << (threadIdx.x & 16);  // the group's lanes
#pragma unroll
  for (int o = 1; o < G; o <<= 1) a = max(a, __shfl_xor_sync(mask, a, o));
  float mul;
  const uint32_t b = h_group_scale<FMT>(a, s, least, tabled, table, mul);
  float w[8] = {};
  w[0] = __fmul_rn(h, mul);
  uint32_t code = fp4::cvt8_e2m1(w) & 15u;
  if (b == fp4::F4<FMT>::kScaleNaN) code = 0;
  const uint32_t next = __shfl_down_sync(mask, code, 1);
  if ((c & 1) == 0) q[c / 2] = static_cast<uint8_t>(code | (next << 4));
  if (c % G == 0) sf[(c / G >> 2) * 512 + (c / G & 3)] = static_cast<uint8_t>(b);
}

// Four (N = 4) or two items of 4 neighbouring elements, 128 columns apart, of every lane. A group of an item is held by 4
// (NVFP4) or 8 lanes. Their maxima are reduced so that every one of four (two) neighbouring lanes ends with another item's,
// makes its scale once for all of them and stores it; likewise each stores the 8 (4) bytes of codes of one item. left:
// columns in the row from the lane's first one on. Bound by the instructions around it: 16384 x 4096 into NVFP4 in 86 us
// (every lane making its groups' scales and storing 16 bits an item: 115; without codes and with h in bf16: 83).
template <int FMT, int N>
__device__ __forceinline__ void emit_items(const Pair* h, int c, int left, float s, uint32_t least, bool tabled, const float* table, uint8_t* q, uint8_t* sf) {
  static_assert(N == 2 || N == 4, "items");
  constexpr uint32_t ALL = 0xFFFFFFFFu;
  constexpr int G = fp4::F4<FMT>::kGroup;
  const int lane = threadIdx.x & 31, j = lane & (N - 1);  // j: the item that this lane ends with
  uint32_t a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 x = split(h[2 * i]), y = split(h[2 * i + 1]);
    a[i] = __float_as_uint(max_nan(max_nan(max_nan(fabsf(x.x), x.y), y.x), y.y));
  }
  uint32_t m;
  if constexpr (N == 4) {
    const bool up = lane & 2;
    const uint32_t k0 = max(up ? a[2] : a[0], __shfl_xor_sync(ALL, up ? a[0] : a[2], 2));
    const uint32_t k1 = max(up ? a[3] : a[1], __shfl_xor_sync(ALL, up ? a[1] : a[3], 2));
    m = max(lane & 1 ? k1 : k0, __shfl_xor_sync(ALL, lane & 1 ? k0 : k1, 1));
  } else {
    m = max(lane & 1 ? a[1] : a[0], __shfl_xor_sync(ALL, lane & 1 ? a[0] : a[1], 1));
    m = max(m, __shfl_xor_sync(ALL, m, 2));
  }
  if constexpr (FMT == 1) m = max(m, __shfl_xor_sync(ALL, m, 4));
  float mul;
  const uint32_t b = h_group_scale<FMT>(m, s, least, tabled, table, mul);
  if (b == fp4::F4<FMT>::kScaleNaN) mul = __uint_as_float(0x7FC00000u);
  const bool mine = 128 * j < left;
  const int g = (c + 128 * j) / G;
  if (mine && (lane & (G / 4 - 1)) < N && (lane & (G / 4 - 1)) == j) sf[(g >> 2) * 512 + (g & 3)] = static_cast<uint8_t>(b);
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = __shfl_sync(ALL, mul, (lane & ~(N - 1)) | i);
    const Pair kk = both(k);
    const float2 x = split(mul2(h[2 * i], kk)), y = split(mul2(h[2 * i + 1], kk));
    w[i] = k == k ? fp4::cvt4_e2m1(x.x, x.y, y.x, y.y) : 0u;
  }
  const int at = (c & ~(4 * N - 1)) + 128 * j;  // the first column of the N lanes' item
  if constexpr (N == 4) {
    // 16 bits of four items in each of four lanes -> four lanes' 16 bits of one item
    const uint32_t lo = __byte_perm(w[0], w[1], 0x5410), hi = __byte_perm(w[2], w[3], 0x5410);
    const bool up = lane & 2;
    const uint32_t other = __shfl_xor_sync(ALL, up ? lo : hi, 2), own = up ? hi : lo;  // two items of lanes l, l ^ 2
    const uint32_t p = up ? other : own, r = up ? own : other;                        // of the lower and of the upper pair
    const uint32_t keep = lane & 1 ? __byte_perm(p, r, 0x7632) : __byte_perm(p, r, 0x5410);
    const uint32_t sent = __shfl_xor_sync(ALL, lane & 1 ? __byte_perm(p, r, 0x5410) : __byte_perm(p, r, 0x7632), 1);
    const uint32_t even = lane & 1 ? sent : keep, odd = lane & 1 ? keep : sent;       // lanes 0, 2 and lanes 1, 3
    if (mine) *reinterpret_cast<uint2*>(q + at / 2) = make_uint2(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
  } else {
    const uint32_t other = __shfl_xor_sync(ALL, lane & 1 ? w[0] : w[1], 1), own = lane & 1 ? w[1] : w[0];
    if (mine) *reinterpret_cast<uint32_t*>(q + at / 2) = lane & 1 ? __byte_perm(other, own, 0x5410) : __byte_perm(own, other, 0x5410);
  }
}

template <int FMT, int VEC, int E>
__device__ __forceinline__ void emit_row(const NormFwd& f, const Pair (&h)[E / 2], int64_t t, int c, int left, const float* table) {
  const float s = h_scale_of(f);
  const bool tabled = s >= 7.888609e-31f && s <= 1.2676506e30f;
  const uint32_t least = fp4::least_scale(s);
  const int width = static_cast<int>(f.width);
  uint8_t *q = f.hq + t * fp4::row_bytes(width), *sf = f.hsf + fp4::scale_offset(t, 0, fp4::atoms_along(FMT, width));
  if constexpr (VEC == 4) {
    constexpr int N = E == 8 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < E / 4; i += N) emit_items<FMT, N>(h + 2 * i, c + 128 * i, left - 128 * i, s, least, tabled, table, q, sf);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float2 a = split(h[i / 2]);
      if (32 * i < left) emit_single<FMT>(i & 1 ? a.y : a.x, c + 32 * i, width, s, least, tabled, table, q, sf);
    }
  }
  // the last atom's groups past the row
  const int groups = width / fp4::F4<FMT>::kGroup;
  const int g = groups + static_cast<int>(threadIdx.x);
  if (g < (groups + 3) / 4 * 4) sf[(g >> 2) * 512 + (g & 3)] = static_cast<uint8_t>(fp4::F4<FMT>::kScaleFill);
}

// The scale atoms' rows past the last token, a word (4 groups) per item; items i, i + stride, ... of this thread.
__device__ __forceinline__ void fill_scales(const NormFwd& f, int64_t i, int64_t stride) {
  const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width);
  const int pad = static_cast<int>((128 - (f.tokens & 127)) & 127);
  for (; i < pad * atoms; i += stride)
    *reinterpret_cast<uint32_t*>(f.hsf + fp4::scale_offset(f.tokens + i / atoms, i % atoms * 4, atoms)) = f.h_fmt == 0 ? 0u : 0x7F7F7F7Fu;
}

}  // namespace norms
}  // namespace fp8gb
