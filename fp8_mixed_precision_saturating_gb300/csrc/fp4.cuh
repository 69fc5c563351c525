// fp4.cuh -- microscaled 4-bit numbers: the group scale rule, the E2M1 cast and the layout of an
// operand's codes and scales (defined in include/fp8gb.h), shared by the quantisers and the norm
// that writes its output in 4 bits.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace fp8gb {
namespace fp4 {

// FMT 0 = NVFP4 (E4M3 scale per 16), 1 = MXFP4 (UE8M0 scale per 32).
template <int FMT>
struct F4 {
  static constexpr int kGroup = FMT == 0 ? 16 : 32;
  static constexpr uint32_t kScaleNaN = FMT == 0 ? 0x7Fu : 0xFFu;
  static constexpr uint32_t kScaleFill = FMT == 0 ? 0u : 127u;  // past the last row or group
};

constexpr float kNvTensorMax = 2688.0f;  // 6 * 448: the largest value under a tensor scale of 1

// Bytes of a row of K codes (whole 16-byte chunks), groups along K, atoms along K.
__host__ __device__ constexpr int64_t row_bytes(int64_t k) { return (k + 31) / 32 * 16; }
__host__ __device__ constexpr int64_t groups_of(int fmt, int64_t k) { return fmt == 0 ? (k + 15) / 16 : (k + 31) / 32; }
__host__ __device__ constexpr int64_t atoms_along(int fmt, int64_t k) { return (groups_of(fmt, k) + 3) / 4; }

// Byte of (row m, group g) in the scale atoms.
__device__ __forceinline__ int64_t scale_offset(int64_t m, int64_t g, int64_t atoms) {
  return ((m >> 7) * atoms + (g >> 2)) * 512 + 16 * (m & 31) + 4 * ((m >> 5) & 3) + (g & 3);
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xFFFFu)));
}

// The value of a UE8M0 byte (0 = 2^-127 is subnormal in fp32; 0xFF is NaN).
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
  return byte == 0u ? __uint_as_float(1u << 22) : byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// fl32(a / 6) for finite a >= 0 where the quotient is normal (below, both round to a zero scale): a product with the
// reciprocal and one residual correction round as the division does (Markstein, 1990), in three instructions.
__device__ __forceinline__ float sixth(float a) {
  const float r = 1.0f / 6.0f, q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-6.0f, q, a), r, q);
}

// The smallest E4M3 code whose value c makes fl32(s / c) finite, for a tensor scale s: the next value above s / 2^128, 1 (2^-9)
// for any s up to 2^118. Under larger ones a group's scale above 0 is raised to it: an infinite factor would make its
// zeros no numbers, where this way its codes still stand for its elements, in larger steps.
__device__ __forceinline__ uint32_t least_scale(float s) {
  const float u = s * 0x1p-64f * 0x1p-64f;
  const uint32_t c = u >= 0x1p-6f ? (__float_as_uint(u) >> 20) - (120u << 3) : static_cast<uint32_t>(u * 512.0f);
  return min(c + 1u, 0x7Eu);
}

// NVFP4's scale byte and factor as group_scale gives them, with the quotients s / 1, s / 1.125, ..., s / 1.875 in
// `table` (filled by quotient) and least_scale(s) in `least`: an E4M3 value is one of those eight times a power of two, so
// fl32(s / c) is an entry times an exact power. (An infinity needs no clamp: the scales that come here are
// at least 2688 / the largest finite bf16, and that has the largest c then too.) A division per group of 16 would be a third of a quantiser's instructions.
__device__ __forceinline__ float quotient(float s, int i) { return __fdiv_rn(s, 1.0f + 0.125f * static_cast<float>(i)); }
__device__ __forceinline__ uint32_t group_scale_nv(uint32_t abits, float s, uint32_t least, const float* table, float& mul) {
  mul = 0.0f;
  if (abits > 0x7F800000u) return 0x7Fu;
  const float t = sixth(fminf(__fmul_rn(__uint_as_float(abits), s), 3.402823466e38f));
  uint16_t e4m3;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e4m3) : "f"(0.0f), "f"(t));
  if (e4m3 == 0) return 0u;
  const uint32_t c = max(static_cast<uint32_t>(e4m3), least), v = __float_as_uint(e4m3_value(c));
  mul = __fmul_rn(table[(v >> 20) & 7u], __uint_as_float((254u << 23) - (v & 0x7F800000u)));
  return c;
}

// The scale byte of a group whose largest magnitude is `a` (fp32 bits `abits`, NaN if the group
// holds one), and the fp32 factor its elements are multiplied by before the cast (0 when they
// are all coded as zero: a zero scale). least: least_scale(s) (NVFP4).
template <int FMT>
__device__ __forceinline__ uint32_t group_scale(uint32_t abits, float s, uint32_t least, float& mul) {
  mul = 0.0f;
  if (abits > 0x7F800000u) return F4<FMT>::kScaleNaN;
  if constexpr (FMT == 0) {
    if (abits == 0x7F800000u) abits = 0x7F7F0000u;  // an infinity counts as the largest finite bf16
    const float t = __fdiv_rn(__fmul_rn(__uint_as_float(abits), s), 6.0f);
    uint16_t e4m3;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e4m3) : "f"(0.0f), "f"(t));
    if (e4m3 == 0) return 0u;
    const uint32_t c = max(static_cast<uint32_t>(e4m3), least);
    mul = __fdiv_rn(s, e4m3_value(c));
    return c;
  } else {
    abits = min(abits, 0x7F7F0000u);  // an infinity counts as the largest finite bf16
    if (abits == 0u) {
      mul = 1.0f;
      return 127u;
    }
    // a = m 2^E with m in [1, 2): 6 2^e = 1.5 2^(e + 2) >= a needs e = E - 2, or E - 1 past 1.5
    int e = static_cast<int>(abits >> 23) - 127 - ((abits & 0x007FFFFFu) <= 0x00400000u ? 2 : 1);
    e = max(e, -127);
    mul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // e <= 126: 2^-e is normal
    return static_cast<uint32_t>(e + 127);
  }
}

// 8 fp32 values -> 8 E2M1 codes, the first in the lowest nibble. Rounds to nearest even and
// saturates; the sign of zero is kept.
__device__ __forceinline__ uint32_t cvt8_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 4 values -> 4 codes in the low 16 bits (and again in the high ones).
__device__ __forceinline__ uint32_t cvt4_e2m1(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "mov.b32 %0, {b0, b1, b0, b1};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}

// 8 codes -> 8 fp32 values.
__device__ __forceinline__ void e2m1_values(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __half2float(__ushort_as_half(static_cast<uint16_t>(h[i] & 0xFFFFu)));
    v[2 * i + 1] = __half2float(__ushort_as_half(static_cast<uint16_t>(h[i] >> 16)));
  }
}

}  // namespace fp4
}  // namespace fp8gb
