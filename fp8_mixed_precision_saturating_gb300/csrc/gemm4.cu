// gemm4.cu -- C = A B^T of two microscaled 4-bit operands.
//
// Formats and layout: include/fp8gb.h, "Microscaled 4-bit operands".
//   C[m, n] = round( d_a d_b sum_g c_a[m, g] c_b[n, g] sum_{k in g} a[m, k] b[n, k] )
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace fp8gb {
namespace {

// One thread per output.
template <int FMT, typename T>
__global__ void __launch_bounds__(256) mm4_kernel(const uint8_t* A, const uint8_t* sfa, const uint8_t* B,
                                                  const uint8_t* sfb, int64_t M, int64_t N, int64_t K, const float* da,
                                                  const float* db, T* C, int64_t ldc) {
  constexpr int G = fp4::F4<FMT>::kGroup;
  pdl_wait();
  pdl_trigger();
  const int64_t n = blockIdx.x * 32ll + (threadIdx.x & 31), atoms = fp4::atoms_along(FMT, K), pitch = fp4::row_bytes(K);
  if (n >= N) return;
  const float d = (da != nullptr ? *da : 1.0f) * (db != nullptr ? *db : 1.0f);
  for (int64_t m = blockIdx.y * 8ll + (threadIdx.x >> 5); m < M; m += gridDim.y * 8ll) {
    float acc = 0.0f;
    for (int64_t g = 0; g * G < K; ++g) {
      const uint32_t ca = sfa[fp4::scale_offset(m, g, atoms)], cb = sfb[fp4::scale_offset(n, g, atoms)];
      const float sa = FMT == 0 ? fp4::e4m3_value(ca) : fp4::ue8m0_value(ca);
      const float sb = FMT == 0 ? fp4::e4m3_value(cb) : fp4::ue8m0_value(cb);
      float p = 0.0f;
      for (int h = 0; h < G / 8; ++h) {
        float a[8], b[8];
        fp4::e2m1_values(*reinterpret_cast<const uint32_t*>(A + m * pitch + g * (G / 2) + 4 * h), a);
        fp4::e2m1_values(*reinterpret_cast<const uint32_t*>(B + n * pitch + g * (G / 2) + 4 * h), b);
        for (int i = 0; i < 8; ++i) p = fmaf(a[i], b[i], p);
      }
      acc = fmaf(p, sa * sb, acc);
    }
    if constexpr (sizeof(T) == 2)
      C[m * ldc + n] = __float2bfloat16_rn(acc * d);
    else
      C[m * ldc + n] = acc * d;
  }
}

template <int FMT, typename T>
cudaError_t launch_as(const Mm4Args& g, cudaStream_t stream) {
  const int64_t rows = (g.M + 7) / 8;
  const dim3 grid(static_cast<unsigned>((g.N + 31) / 32), static_cast<unsigned>(rows < 65535 ? rows : 65535));
  return launch_pdl(mm4_kernel<FMT, T>, grid, dim3(256), 0, stream, static_cast<const uint8_t*>(g.A),
                    static_cast<const uint8_t*>(g.sfa), static_cast<const uint8_t*>(g.B),
                    static_cast<const uint8_t*>(g.sfb), g.M, g.N, g.K, g.da, g.db, static_cast<T*>(g.C), g.ldc);
}

}  // namespace

cudaError_t launch_mm4(const Mm4Args& g, cudaStream_t stream, const char** why) {
  (void)why;
  if (g.f32) return g.fmt == 0 ? launch_as<0, float>(g, stream) : launch_as<1, float>(g, stream);
  return g.fmt == 0 ? launch_as<0, __nv_bfloat16>(g, stream) : launch_as<1, __nv_bfloat16>(g, stream);
}

}  // namespace fp8gb
