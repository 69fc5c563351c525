// norm.cu -- the norms around a block with its gate and the residual's scale, forward and backward.
//
//   n = norm_post(o) w_post + b_post;  r' = alpha r + gate n;  h = norm_pre(r') w_pre + b_pre
//
// (include/fp8gb.h, "The norms around a block"). Every norm is z = (x - mean) rstd, then z w + b.
// Backward, with g the gradient at r' and D the width:
//   norm'(dy; x):  dz = dy w,  dx = rstd (dz - z mean(dz z) - [layer] mean(dz)),
//                  dw = sum_t dy z,  db = sum_t dy
//   g = dr_out + norm_pre'(dh; r');  dr = alpha g;  dalpha = sum g r
//   dn = gate g;  dgate = sum over the gate's rows of g n;  do = norm_post'(dn; o)
// Statistics and sums are held in fp32; a layer norm's variance is taken about its mean (two
// passes over the row), so a large mean does not cancel it away.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace fp8gb {
namespace {

constexpr int kNone = 0, kRms = 1, kLayer = 2;
constexpr int THREADS = 256;

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Sums of two values over the CTA, the same bits on every thread.
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  __syncthreads();  // the previous sum's values have been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    s.x += red[w].x;
    s.y += red[w].y;
  }
  return s;
}

// Mean and 1 / root of a row whose element c is value(c).
template <typename F>
__device__ __forceinline__ float2 row_stat(int kind, int64_t width, float eps, float2* red, F value) {
  float2 st = make_float2(0.0f, 1.0f);
  if (kind == kNone) return st;
  const float n = static_cast<float>(width);
  if (kind == kLayer) {
    float a = 0.0f;
    for (int64_t c = threadIdx.x; c < width; c += THREADS) a += value(c);
    st.x = block_sum(a, 0.0f, red).x / n;
  }
  float a = 0.0f;
  for (int64_t c = threadIdx.x; c < width; c += THREADS) {
    const float z = value(c) - st.x;
    a = fmaf(z, z, a);
  }
  st.y = 1.0f / sqrtf(block_sum(a, 0.0f, red).x / n + eps);
  return st;
}

__device__ __forceinline__ float affine(float z, const float* w, const float* b, int64_t c) {
  if (w != nullptr) z *= w[c];
  return b != nullptr ? z + b[c] : z;
}

// One CTA per token, the row read again for every pass over it.
template <typename TS, typename TB>
__global__ void __launch_bounds__(THREADS) norm_fwd_kernel(const NormFwd f) {
  __shared__ float2 red[THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float alpha = f.res_scale != nullptr ? *f.res_scale : 1.0f;
  for (int64_t t = blockIdx.x; t < f.tokens; t += gridDim.x) {
    const TS* r = static_cast<const TS*>(f.r) + t * f.ld_r;
    const TB* o = f.o != nullptr ? static_cast<const TB*>(f.o) + t * f.ld_o : nullptr;
    const TB* gate = f.gate != nullptr ? static_cast<const TB*>(f.gate) + t / f.gate_rows * f.ld_gate : nullptr;
    const float2 post = row_stat(f.post, f.width, f.eps, red, [&](int64_t c) { return load(o + c); });
    auto mid = [&](int64_t c) {
      float v = load(r + c) * alpha;
      if (o == nullptr) return v;
      const float n = affine((load(o + c) - post.x) * post.y, f.w_post, f.b_post, c);
      return gate != nullptr ? fmaf(load(gate + c), n, v) : v + n;
    };
    const float2 pre = row_stat(f.pre, f.width, f.eps, red, mid);
    if (threadIdx.x == 0) {
      if (f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = post;
      if (f.stat_pre != nullptr) reinterpret_cast<float2*>(f.stat_pre)[t] = pre;
    }
    // each thread reads its columns before it writes them, so r_out may be r
    for (int64_t c = threadIdx.x; c < f.width; c += THREADS) {
      const float m = mid(c);
      const float h = affine((m - pre.x) * pre.y, f.w_pre, f.b_pre, c);
      if (f.h != nullptr) store(static_cast<TB*>(f.h) + t * f.ld_h + c, h);
      if (f.hq == nullptr && f.r_out != nullptr) store(static_cast<TS*>(f.r_out) + t * f.ld_r_out + c, m);
    }
    if (f.hq != nullptr) {
      const float s = f.h_scale != nullptr ? *f.h_scale : 1.0f;
      const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width), pitch = fp4::row_bytes(f.width);
      const int group = f.h_fmt == 0 ? 16 : 32;
      for (int64_t g = threadIdx.x; g < f.width / group; g += THREADS) {
        uint32_t a = 0;
        auto hv = [&](int64_t c) { return affine((mid(c) - pre.x) * pre.y, f.w_pre, f.b_pre, c); };
        for (int i = 0; i < group; ++i) a = max(a, __float_as_uint(hv(g * group + i)) & 0x7FFFFFFFu);
        float mul;
        const uint32_t b = f.h_fmt == 0 ? fp4::group_scale<0>(a, s, mul) : fp4::group_scale<1>(a, s, mul);
        f.hsf[fp4::scale_offset(t, g, atoms)] = static_cast<uint8_t>(b);
        for (int i = 0; i < group; i += 8) {
          float w[8];
          for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(hv(g * group + i + j), mul);
          const bool nan = a > 0x7F800000u;
          *reinterpret_cast<uint32_t*>(f.hq + t * pitch + (g * group + i) / 2) = nan ? 0u : fp4::cvt8_e2m1(w);
        }
      }
      __syncthreads();
      if (f.r_out != nullptr)
        for (int64_t c = threadIdx.x; c < f.width; c += THREADS)
          store(static_cast<TS*>(f.r_out) + t * f.ld_r_out + c, mid(c));
    }
  }
  if (f.hq != nullptr) {  // the atoms' padding: rows past the last token, groups past the last
    const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width), groups = fp4::groups_of(f.h_fmt, f.width);
    const int64_t mpad = (f.tokens + 127) / 128 * 128, n = mpad * atoms * 4;
    const uint8_t fill = f.h_fmt == 0 ? 0 : 127;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * THREADS) {
      const int64_t m = i / (atoms * 4), g = i - m * (atoms * 4);
      if (m >= f.tokens || g >= groups) f.hsf[fp4::scale_offset(m, g, atoms)] = fill;
    }
  }
}

// ---------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------
// CTA p takes the consecutive tokens [p R, (p + 1) R) and keeps its share of every column sum in
// its own rows of the workspace: 4 rows for the parameters, then 2 for the gate gradient of the
// groups that it shares with its neighbours (its first group, its last). A group inside one CTA's
// tokens is written out by that CTA alone.
constexpr int kPart = 6;

template <typename TS, typename TB>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(const NormFwd f, const NormBwd b, float* part, double* part_alpha,
                                                           int64_t rows_per) {
  __shared__ float2 red[THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float alpha = f.res_scale != nullptr ? *f.res_scale : 1.0f;
  const int64_t D = f.width, t0 = blockIdx.x * rows_per, t1 = min(t0 + rows_per, f.tokens);
  const float inv = 1.0f / static_cast<float>(D);
  float* mine = part + static_cast<int64_t>(blockIdx.x) * kPart * D;
  for (int64_t c = threadIdx.x; c < kPart * D; c += THREADS) mine[c] = 0.0f;
  // sum g r cancels (its terms have both signs): the row's share in fp32, the rows in fp64
  double dalpha = 0.0;
  for (int64_t t = t0; t < t1; ++t) {
    float row_alpha = 0.0f;
    const TS* rp = f.r_out != nullptr ? static_cast<const TS*>(f.r_out) + t * f.ld_r_out : nullptr;
    const TS* r = f.r != nullptr ? static_cast<const TS*>(f.r) + t * f.ld_r : nullptr;
    const TB* o = f.o != nullptr ? static_cast<const TB*>(f.o) + t * f.ld_o : nullptr;
    const TB* dh = b.dh != nullptr ? static_cast<const TB*>(b.dh) + t * b.ld_dh : nullptr;
    const TS* dro = b.dr_out != nullptr ? static_cast<const TS*>(b.dr_out) + t * b.ld_dr_out : nullptr;
    const int64_t grp = f.gate != nullptr ? t / f.gate_rows : 0;
    const TB* gate = f.gate != nullptr ? static_cast<const TB*>(f.gate) + grp * f.ld_gate : nullptr;
    const float2 pre = f.pre != kNone && dh != nullptr ? reinterpret_cast<const float2*>(f.stat_pre)[t] : make_float2(0.0f, 1.0f);
    const float2 post = f.post != kNone ? reinterpret_cast<const float2*>(f.stat_post)[t] : make_float2(0.0f, 1.0f);
    float2 s1 = make_float2(0.0f, 0.0f);
    auto zpre = [&](int64_t c) { return f.pre != kNone ? (load(rp + c) - pre.x) * pre.y : 0.0f; };
    if (f.pre != kNone && dh != nullptr) {
      float a = 0.0f, q = 0.0f;
      for (int64_t c = threadIdx.x; c < D; c += THREADS) {
        const float dz = f.w_pre != nullptr ? load(dh + c) * f.w_pre[c] : load(dh + c);
        a += dz;
        q = fmaf(dz, zpre(c), q);
      }
      s1 = block_sum(a, q, red);
    }
    auto grad = [&](int64_t c) {
      float g = dro != nullptr ? load(dro + c) : 0.0f;
      if (dh == nullptr) return g;
      const float dy = load(dh + c);
      if (f.pre == kNone) return g + dy;
      const float dz = f.w_pre != nullptr ? dy * f.w_pre[c] : dy;
      float dx = dz - zpre(c) * (s1.y * inv);
      if (f.pre == kLayer) dx -= s1.x * inv;
      return fmaf(dx, pre.y, g);
    };
    float2 s2 = make_float2(0.0f, 0.0f);
    if (f.post != kNone) {
      float a = 0.0f, q = 0.0f;
      for (int64_t c = threadIdx.x; c < D; c += THREADS) {
        float dz = grad(c);
        if (gate != nullptr) dz *= load(gate + c);
        if (f.w_post != nullptr) dz *= f.w_post[c];
        a += dz;
        q = fmaf(dz, (load(o + c) - post.x) * post.y, q);
      }
      s2 = block_sum(a, q, red);
    }
    const bool whole = f.gate != nullptr && grp * f.gate_rows >= t0 && (min((grp + 1) * f.gate_rows, f.tokens) <= t1);
    const bool last = f.gate != nullptr && (t + 1 == t1 || (t + 1) / f.gate_rows != grp);
    const int slot = f.gate != nullptr && grp != t0 / f.gate_rows ? 5 : 4;
    for (int64_t c = threadIdx.x; c < D; c += THREADS) {
      const float g = grad(c);
      if (dh != nullptr) {
        const float dy = load(dh + c);
        mine[c] = fmaf(dy, zpre(c), mine[c]);
        mine[D + c] += dy;
      }
      if (b.dres_scale != nullptr) row_alpha = fmaf(g, load(r + c), row_alpha);
      if (o != nullptr) {
        const float z = (load(o + c) - post.x) * post.y;
        const float dn = gate != nullptr ? g * load(gate + c) : g;
        mine[2 * D + c] = fmaf(dn, z, mine[2 * D + c]);
        mine[3 * D + c] += dn;
        if (b.dgate != nullptr) {
          float* acc = mine + slot * D + c;
          const float v = fmaf(g, affine(z, f.w_post, f.b_post, c), *acc);
          *acc = v;
          if (last && whole) {
            b.dgate[grp * D + c] = v;
            *acc = 0.0f;
          }
        }
        float dx = dn;
        if (f.post != kNone) {
          const float dz = f.w_post != nullptr ? dn * f.w_post[c] : dn;
          dx = dz - z * (s2.y * inv);
          if (f.post == kLayer) dx -= s2.x * inv;
          dx *= post.y;
        }
        if (b.dO != nullptr) store(static_cast<TB*>(b.dO) + t * b.ld_do + c, dx);
      }
      if (b.dr != nullptr) store(static_cast<TS*>(b.dr) + t * b.ld_dr + c, g * alpha);
    }
    dalpha += row_alpha;
  }
  if (b.dres_scale != nullptr) {
    __shared__ double sums[THREADS];
    sums[threadIdx.x] = dalpha;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int i = 0; i < THREADS; ++i) s += sums[i];
      part_alpha[blockIdx.x] = s;
    }
  }
}

// Column sums over the CTAs' partial rows, in CTA order. blockIdx.y 0: the parameters and alpha;
// blockIdx.y = p > 0: the gate group that CTAs p - 1 and p share, if CTA p - 1 holds its first token.
__global__ void __launch_bounds__(THREADS) norm_bwd_reduce_kernel(const NormFwd f, const NormBwd b, const float* part,
                                                                  const double* part_alpha, int64_t rows_per, int ctas) {
  pdl_wait();
  pdl_trigger();
  const int64_t D = f.width, c = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x;
  if (blockIdx.y == 0) {
    if (c < D) {
      float* out[4] = {b.dw_pre, b.db_pre, b.dw_post, b.db_post};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (out[k] == nullptr) continue;
        float s = 0.0f;
        for (int p = 0; p < ctas; ++p) s += part[(static_cast<int64_t>(p) * kPart + k) * D + c];
        out[k][c] = s;
      }
    }
    if (b.dres_scale != nullptr && blockIdx.x == 0 && threadIdx.x == 0) {
      double s = 0.0;
      for (int p = 0; p < ctas; ++p) s += part_alpha[p];
      *b.dres_scale = static_cast<float>(s);
    }
    return;
  }
  for (int p = blockIdx.y; p < ctas; p += gridDim.y - 1) {
    const int64_t first = p * rows_per;  // CTA p's first token
    const int64_t grp = first / f.gate_rows, ga = grp * f.gate_rows, ge = min(ga + f.gate_rows, f.tokens);
    if (ga == first || ga / rows_per != p - 1 || c >= D) continue;
    float s = 0.0f;
    for (int64_t q = p - 1; q * rows_per < ge; ++q) {
      const int slot = (q * rows_per) / f.gate_rows == grp ? 4 : 5;
      s += part[(q * kPart + slot) * D + c];
    }
    b.dgate[grp * D + c] = s;
  }
}

struct BwdPlan {
  int ctas;
  int64_t rows_per;
};

BwdPlan bwd_plan(int64_t tokens) {
  const int64_t most = 2ll * num_sms();
  const int64_t rows = (tokens + most - 1) / most;
  return {static_cast<int>((tokens + rows - 1) / rows), rows};
}

template <typename TS, typename TB>
cudaError_t bwd_as(const NormFwd& f, const NormBwd& b, void* ws, cudaStream_t stream) {
  const BwdPlan pl = bwd_plan(f.tokens);
  double* part_alpha = static_cast<double*>(ws);
  float* part = reinterpret_cast<float*>(part_alpha + pl.ctas + (pl.ctas & 1));
  cudaError_t e = launch_pdl(norm_bwd_kernel<TS, TB>, dim3(pl.ctas), dim3(THREADS), 0, stream, f, b, part, part_alpha, pl.rows_per);
  if (e != cudaSuccess) return e;
  const bool split = b.dgate != nullptr && pl.ctas > 1;
  const dim3 grid(static_cast<unsigned>((f.width + THREADS - 1) / THREADS), split ? static_cast<unsigned>(pl.ctas) : 1u);
  return launch_pdl(norm_bwd_reduce_kernel, grid, dim3(THREADS), 0, stream, f, b, part, part_alpha, pl.rows_per, pl.ctas);
}

template <typename TS, typename TB>
cudaError_t fwd_as(const NormFwd& f, cudaStream_t stream) {
  const int64_t most = 8ll * num_sms();
  return launch_pdl(norm_fwd_kernel<TS, TB>, dim3(static_cast<unsigned>(f.tokens < most ? f.tokens : most)), dim3(THREADS), 0, stream, f);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& f, cudaStream_t stream) {
  if (f.stream_f32)
    return f.block_f32 ? fwd_as<float, float>(f, stream) : fwd_as<float, __nv_bfloat16>(f, stream);
  return f.block_f32 ? fwd_as<__nv_bfloat16, float>(f, stream) : fwd_as<__nv_bfloat16, __nv_bfloat16>(f, stream);
}

int64_t norm_bwd_workspace_bytes(const NormFwd& f) {
  if (f.tokens == 0 || f.width == 0) return 0;
  const int64_t ctas = bwd_plan(f.tokens).ctas;
  return ctas * kPart * f.width * 4 + (ctas + 1) / 2 * 16;
}

cudaError_t launch_norm_bwd(const NormFwd& f, const NormBwd& b, void* ws, cudaStream_t stream) {
  if (f.stream_f32)
    return f.block_f32 ? bwd_as<float, float>(f, b, ws, stream) : bwd_as<float, __nv_bfloat16>(f, b, ws, stream);
  return f.block_f32 ? bwd_as<__nv_bfloat16, float>(f, b, ws, stream) : bwd_as<__nv_bfloat16, __nv_bfloat16>(f, b, ws, stream);
}

}  // namespace fp8gb
