// quant4.cu -- bf16 matrices into microscaled 4-bit operands and back (HBM-bound kernels).
//
// Formats, scale rule and layout: include/fp8gb.h, "Microscaled 4-bit operands".
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cast.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace fp8gb {
namespace {

using namespace castops;

// The tensor scale of a call: 1 without a state, else from the state's amax or history; the
// first thread of the grid records it.
__device__ __forceinline__ float tensor_scale(const QuantState& st, bool delayed, bool first) {
  if (st.scale == nullptr) return 1.0f;
  float s, d;
  scales_from_amax(effective_amax(st, delayed), fp4::kNvTensorMax, s, d);
  if (first) {
    *st.scale = s;
    *st.scale_inv = d;
  }
  return s;
}

// max |x| of a matrix onto *st.amax_cur. In delayed mode only while the history is empty (later
// casts take the scale from the history and this kernel's maximum with it).
__global__ void amax4_kernel(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, QuantState st, int record) {
  pdl_wait();
  pdl_trigger();
  (void)record;
  uint32_t m = 0;
  const int64_t n = rows * cols;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / cols;
    const uint32_t b = x[r * ld + (i - r * cols)] & 0x7FFFu;
    if (b <= 0x7F80u) m = max(m, b);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) atomic_max_amax(st.amax_cur, m);
}

// One thread per (row, group) of the operand, its padding included. DOWN: the operand's rows are
// x's columns.
template <int FMT, bool DOWN>
__global__ void __launch_bounds__(256) quant4_kernel(const uint16_t* x, int64_t mn, int64_t k, int64_t ld,
                                                     QuantState st, int delayed, uint8_t* q, uint8_t* sf) {
  constexpr int G = fp4::F4<FMT>::kGroup;
  pdl_wait();
  pdl_trigger();
  const float s = tensor_scale(st, delayed != 0, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  const int64_t atoms = fp4::atoms_along(FMT, k), pitch = fp4::row_bytes(k);
  const int64_t m = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (m >= (mn + 127) / 128 * 128) return;
  for (int64_t g = blockIdx.y; g < atoms * 4; g += gridDim.y) {
    uint32_t scale = fp4::F4<FMT>::kScaleFill;
    float v[G];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int64_t c = g * G + i;
      uint32_t b = 0;
      if (m < mn && c < k) b = static_cast<uint32_t>(DOWN ? x[c * ld + m] : x[m * ld + c]) << 16;
      v[i] = __uint_as_float(b);
      a = max(a, b & 0x7FFFFFFFu);
    }
    float mul = 0.0f;
    if (m < mn && g * G < k) scale = fp4::group_scale<FMT>(a, s, mul);
    sf[fp4::scale_offset(m, g, atoms)] = static_cast<uint8_t>(scale);
    if (m < mn && g * (G / 2) < pitch) {
#pragma unroll
      for (int h = 0; h < G / 8; ++h) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __fmul_rn(v[8 * h + i], mul);
        const uint32_t c = scale == fp4::F4<FMT>::kScaleNaN ? 0u : fp4::cvt8_e2m1(w);
        *reinterpret_cast<uint32_t*>(q + m * pitch + g * (G / 2) + 4 * h) = c;
      }
    }
  }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(256) dequant4_kernel(const uint8_t* q, const uint8_t* sf, int64_t mn, int64_t k,
                                                       const float* scale_inv, T* y, int64_t ldy) {
  constexpr int G = fp4::F4<FMT>::kGroup;
  pdl_wait();
  pdl_trigger();
  const float d = scale_inv != nullptr ? *scale_inv : 1.0f;
  const int64_t atoms = fp4::atoms_along(FMT, k), pitch = fp4::row_bytes(k), words = (k + 7) / 8;
  const int64_t n = mn * words;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t m = i / words, w = i - m * words;
    const uint32_t b = sf[fp4::scale_offset(m, w * 8 / G, atoms)];
    const float c = FMT == 0 ? fp4::e4m3_value(b) : fp4::ue8m0_value(b);
    float v[8];
    fp4::e2m1_values(*reinterpret_cast<const uint32_t*>(q + m * pitch + 4 * w), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (8 * w + j >= k) break;
      const float f = __fmul_rn(__fmul_rn(v[j], c), d);
      if constexpr (sizeof(T) == 2)
        y[m * ldy + 8 * w + j] = __float2bfloat16_rn(f);
      else
        y[m * ldy + 8 * w + j] = f;
    }
  }
}

template <int FMT, bool DOWN>
cudaError_t launch_one(const void* x, int64_t mn, int64_t k, int64_t ld, const QuantState& st, bool delayed, void* q,
                       void* sf, cudaStream_t stream) {
  const int64_t groups = fp4::atoms_along(FMT, k) * 4;
  const dim3 grid(static_cast<unsigned>((mn + 255) / 256), static_cast<unsigned>(groups < 65535 ? groups : 65535));
  return launch_pdl(quant4_kernel<FMT, DOWN>, grid, dim3(256), 0, stream, static_cast<const uint16_t*>(x), mn, k, ld, st,
                    delayed ? 1 : 0, static_cast<uint8_t*>(q), static_cast<uint8_t*>(sf));
}

}  // namespace

cudaError_t launch_quant4(int fmt, bool delayed, const void* x, int64_t rows, int64_t cols, int64_t ld,
                          const QuantState& st, void* q, void* sf, void* qT, void* sfT, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (st.scale != nullptr) {
    if (!delayed && (e = cudaMemsetAsync(st.amax_cur, 0, sizeof(float), stream)) != cudaSuccess) return e;
    e = launch_pdl(amax4_kernel, dim3(8 * num_sms()), dim3(256), 0, stream, static_cast<const uint16_t*>(x), rows, cols,
                   ld, st, delayed ? 1 : 0);
    if (e != cudaSuccess) return e;
  }
  if (q != nullptr) {
    e = fmt == 0 ? launch_one<0, false>(x, rows, cols, ld, st, delayed, q, sf, stream)
                 : launch_one<1, false>(x, rows, cols, ld, st, delayed, q, sf, stream);
    if (e != cudaSuccess) return e;
  }
  if (qT != nullptr)
    e = fmt == 0 ? launch_one<0, true>(x, cols, rows, ld, st, delayed, qT, sfT, stream)
                 : launch_one<1, true>(x, cols, rows, ld, st, delayed, qT, sfT, stream);
  return e;
}

cudaError_t launch_dequant4(int fmt, bool f32, const void* q, const void* sf, int64_t mn, int64_t k,
                            const float* scale_inv, void* y, int64_t ldy, cudaStream_t stream) {
  const int64_t n = mn * ((k + 7) / 8);
  const int64_t want = (n + 255) / 256, most = 16ll * num_sms();
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  const uint8_t* qb = static_cast<const uint8_t*>(q);
  const uint8_t* sb = static_cast<const uint8_t*>(sf);
  if (f32)
    return fmt == 0 ? launch_pdl(dequant4_kernel<0, float>, grid, dim3(256), 0, stream, qb, sb, mn, k, scale_inv, static_cast<float*>(y), ldy)
                    : launch_pdl(dequant4_kernel<1, float>, grid, dim3(256), 0, stream, qb, sb, mn, k, scale_inv, static_cast<float*>(y), ldy);
  return fmt == 0 ? launch_pdl(dequant4_kernel<0, __nv_bfloat16>, grid, dim3(256), 0, stream, qb, sb, mn, k, scale_inv, static_cast<__nv_bfloat16*>(y), ldy)
                  : launch_pdl(dequant4_kernel<1, __nv_bfloat16>, grid, dim3(256), 0, stream, qb, sb, mn, k, scale_inv, static_cast<__nv_bfloat16*>(y), ldy);
}

}  // namespace fp8gb
