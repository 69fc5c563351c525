// norm_emit.cuh -- what the forward kernels of the norms share beyond norm.cuh: h in 4 bits, and the choice of the
// kernel for many rows.
#pragma once
#include "fp4.cuh"
#include "norm.cuh"

namespace fp8gb {

// Many rows of whole 16 bytes with a block's output (norm_fwd_ring.cu); taken: whether it was one for that kernel.
cudaError_t launch_norm_fwd_ring(const NormFwd& f, cudaStream_t stream, bool* taken);

namespace norms {

inline uint32_t gate_rows_of(const NormFwd& f) { return static_cast<uint32_t>(f.gate == nullptr || f.gate_rows > f.tokens ? f.tokens : f.gate_rows); }

// The quotients that NVFP4's group factors are made of (fp4::quotient), by 8 threads; the caller puts a barrier before emit_row.
__device__ __forceinline__ float h_scale_of(const NormFwd& f) { return f.h_scale != nullptr ? __ldg(f.h_scale) : 1.0f; }
__device__ __forceinline__ void fill_table(const NormFwd& f, float* table, int tid) {
  if (f.hq != nullptr && f.h_fmt == 0 && tid < 8) table[tid] = fp4::quotient(h_scale_of(f), tid);
}

// VEC consecutive elements of h as 4-bit codes, with their group's scale (16 or 32 neighbouring elements, held by
// neighbouring lanes, all of them in the row: width % 32 == 0). q, sf: the row's codes, and its byte of group 0 in the
// scale atoms. The caller's tensor scale may be any number: outside [2^-100, 2^100] the quotients could round where
// the division does not, so it is divided then (tabled: not). 16384 x 4096 into NVFP4, divided 119 us.
template <int FMT, int VEC>
__device__ __forceinline__ void emit_codes(const float (&h)[VEC], int c, int width, float s, bool tabled, const float* table, uint8_t* q, uint8_t* sf) {
  constexpr int G = fp4::F4<FMT>::kGroup, LANES = G / VEC;
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) a = max(a, __float_as_uint(h[j]) & 0x7FFFFFFFu);
  const uint32_t mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));  // the group's lanes
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) a = max(a, __shfl_xor_sync(mask, a, o));
  float mul;
  uint32_t b;
  if constexpr (FMT == 0)
    b = tabled ? fp4::group_scale_nv(a, s, table, mul) : fp4::group_scale<FMT>(a, s, mul);
  else
    b = fp4::group_scale<FMT>(a, s, mul);
  float w[8] = {};
#pragma unroll
  for (int j = 0; j < VEC; ++j) w[j] = __fmul_rn(h[j], mul);
  uint32_t codes = fp4::cvt8_e2m1(w);
  if (b == fp4::F4<FMT>::kScaleNaN) codes = 0;
  if constexpr (VEC == 4) {
    *reinterpret_cast<uint16_t*>(q + c / 2) = static_cast<uint16_t>(codes);
  } else {
    const uint32_t next = __shfl_down_sync(mask, codes, 1);
    if ((c & 1) == 0) q[c / 2] = static_cast<uint8_t>((codes & 15u) | (next << 4));
  }
  if (c % G == 0) {
    const int g = c / G;
    uint8_t* at = sf + (g >> 2) * 512;
    at[g & 3] = static_cast<uint8_t>(b);
    if (c + G >= width)  // the last atom's groups past the row
      for (int e = g + 1; (e & 3) != 0; ++e) at[e & 3] = static_cast<uint8_t>(fp4::F4<FMT>::kScaleFill);
  }
}

template <int FMT, int VEC, int E>
__device__ __forceinline__ void emit_row(const NormFwd& f, const Pair (&h)[E / 2], int64_t t, int c, int left, const float* table) {
  const float s = h_scale_of(f);
  const bool tabled = s >= 7.888609e-31f && s <= 1.2676506e30f;
  const int width = static_cast<int>(f.width);
  uint8_t *q = f.hq + t * fp4::row_bytes(width), *sf = f.hsf + fp4::scale_offset(t, 0, fp4::atoms_along(FMT, width));
#pragma unroll
  for (int i = 0; i < E / VEC; ++i) {
    if (32 * VEC * i < left) {
      float v[VEC];
      if constexpr (VEC == 4) {
        const float2 a = split(h[2 * i]), b = split(h[2 * i + 1]);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
      } else {
        const float2 a = split(h[i / 2]);
        v[0] = i & 1 ? a.y : a.x;
      }
      emit_codes<FMT, VEC>(v, c + 32 * VEC * i, width, s, tabled, table, q, sf);
    }
  }
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
