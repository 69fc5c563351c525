// norm_fwd.cu -- forward of the norms around a block with its gate and the residual's scale (HBM-bound).
#include "fp4.cuh"
#include "norm.cuh"

namespace fp8gb {
namespace {

using namespace norms;

// Mean and 1 / root of a row whose element c is value(c).
template <typename F>
__device__ __forceinline__ float2 row_stat(int kind, int64_t width, float eps, float2 (*red)[32], int& turn, F value) {
  float2 st = make_float2(0.0f, 1.0f);
  if (kind == kNone) return st;
  const float n = static_cast<float>(width);
  if (kind == kLayer) {
    float a = 0.0f;
    for (int64_t c = threadIdx.x; c < width; c += kThreads) a += value(c);
    st.x = cta_sum2(make_float2(a, 0.0f), red, turn, kThreads / 32).x / n;
  }
  float a = 0.0f;
  for (int64_t c = threadIdx.x; c < width; c += kThreads) {
    const float z = value(c) - st.x;
    a = fmaf(z, z, a);
  }
  st.y = 1.0f / sqrtf(cta_sum2(make_float2(a, 0.0f), red, turn, kThreads / 32).x / n + eps);
  return st;
}

// Any width and alignment: one CTA per token, the row read again for every pass over it.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) norm_fwd_any_kernel(const NormFwd f) {
  __shared__ float2 red[2][32];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const float alpha = f.res_scale != nullptr ? *f.res_scale : 1.0f;
  for (int64_t t = blockIdx.x; t < f.tokens; t += gridDim.x) {
    const TS* r = static_cast<const TS*>(f.r) + t * f.ld_r;
    const TB* o = f.o != nullptr ? static_cast<const TB*>(f.o) + t * f.ld_o : nullptr;
    const TB* gate = f.gate != nullptr ? static_cast<const TB*>(f.gate) + t / f.gate_rows * f.ld_gate : nullptr;
    const float2 post = row_stat(f.post, f.width, f.eps, red, turn, [&](int64_t c) { return load(o + c); });
    auto mid = [&](int64_t c) {
      float v = load(r + c) * alpha;
      if (o == nullptr) return v;
      const float n = affine((load(o + c) - post.x) * post.y, f.w_post, f.b_post, c);
      return gate != nullptr ? fmaf(load(gate + c), n, v) : v + n;
    };
    const float2 pre = row_stat(f.pre, f.width, f.eps, red, turn, mid);
    if (threadIdx.x == 0) {
      if (f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = post;
      if (f.stat_pre != nullptr) reinterpret_cast<float2*>(f.stat_pre)[t] = pre;
    }
    // each thread reads its columns before it writes them, so r_out may be r
    for (int64_t c = threadIdx.x; c < f.width; c += kThreads) {
      const float m = mid(c);
      const float h = affine((m - pre.x) * pre.y, f.w_pre, f.b_pre, c);
      if (f.h != nullptr) store(static_cast<TB*>(f.h) + t * f.ld_h + c, h);
      if (f.hq == nullptr && f.r_out != nullptr) store(static_cast<TS*>(f.r_out) + t * f.ld_r_out + c, m);
    }
    if (f.hq != nullptr) {
      const float s = f.h_scale != nullptr ? *f.h_scale : 1.0f;
      const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width), pitch = fp4::row_bytes(f.width);
      const int group = f.h_fmt == 0 ? 16 : 32;
      for (int64_t g = threadIdx.x; g < f.width / group; g += kThreads) {
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
        for (int64_t c = threadIdx.x; c < f.width; c += kThreads)
          store(static_cast<TS*>(f.r_out) + t * f.ld_r_out + c, mid(c));
    }
  }
  if (f.hq != nullptr) {  // the atoms' padding: rows past the last token, groups past the last
    const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width), groups = fp4::groups_of(f.h_fmt, f.width);
    const int64_t mpad = (f.tokens + 127) / 128 * 128, n = mpad * atoms * 4;
    const uint8_t fill = f.h_fmt == 0 ? 0 : 127;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
      const int64_t m = i / (atoms * 4), g = i - m * (atoms * 4);
      if (m >= f.tokens || g >= groups) f.hsf[fp4::scale_offset(m, g, atoms)] = fill;
    }
  }
}

// ---------------------------------------------------------------------------------------
// A row in the registers of its warps
// ---------------------------------------------------------------------------------------
// The row's elements are read once and stay in registers through both statistics. `blockDim.x / 32` warps share
// a row, a lane holds I items of VEC consecutive elements (item i of thread x starts at column
// (i blockDim.x + x) VEC, so every access of a warp is contiguous); a warp that holds a whole row needs no
// barrier, and blockDim.y such rows share a CTA. The parameters come from L1, where the streamed rows do not
// displace them.
template <int VEC, int I>
__device__ __forceinline__ float2 held_stat(int kind, int width, float eps, const float (&v)[I][VEC], float2 (*red)[32], int& turn) {
  float2 st = make_float2(0.0f, 1.0f);
  if (kind == kNone) return st;
  const int warps = blockDim.x >> 5;
  const float n = static_cast<float>(width);
  if (kind == kLayer) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < I; ++i)  // (elements past the row are zero)
#pragma unroll
      for (int j = 0; j < VEC; ++j) a += v[i][j];
    st.x = cta_sum2(make_float2(a, 0.0f), red, turn, warps).x / n;
  }
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const bool in = static_cast<int>(i * blockDim.x + threadIdx.x) * VEC < width;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float z = in ? v[i][j] - st.x : 0.0f;
      a = fmaf(z, z, a);
    }
  }
  st.y = 1.0f / sqrtf(cta_sum2(make_float2(a, 0.0f), red, turn, warps).x / n + eps);
  return st;
}

// An item of h as 4-bit codes, with its group's scale (the group is 16 or 32 neighbouring elements, held by
// neighbouring lanes, all of them in the row: width % 32 == 0).
template <int FMT, int VEC>
__device__ __forceinline__ void emit_codes(const NormFwd& f, const float (&h)[VEC], int64_t t, int c, float s, int64_t pitch, int64_t atoms) {
  constexpr int G = fp4::F4<FMT>::kGroup, LANES = G / VEC;
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) a = max(a, __float_as_uint(h[j]) & 0x7FFFFFFFu);
  const uint32_t mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));  // the group's lanes
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) a = max(a, __shfl_xor_sync(mask, a, o));
  float mul;
  const uint32_t b = fp4::group_scale<FMT>(a, s, mul);
  const bool nan = b == fp4::F4<FMT>::kScaleNaN;
  float w[8] = {};
#pragma unroll
  for (int j = 0; j < VEC; ++j) w[j] = __fmul_rn(h[j], mul);
  uint32_t codes = fp4::cvt8_e2m1(w);
  if (nan) codes = 0;
  if constexpr (VEC == 4) {
    *reinterpret_cast<uint16_t*>(f.hq + t * pitch + c / 2) = static_cast<uint16_t>(codes);
  } else {
    const uint32_t next = __shfl_down_sync(mask, codes, 1);
    if ((c & 1) == 0) f.hq[t * pitch + c / 2] = static_cast<uint8_t>((codes & 15u) | (next << 4));
  }
  if (c % G == 0) {
    const int g = c / G;
    f.hsf[fp4::scale_offset(t, g, atoms)] = static_cast<uint8_t>(b);
    if (c + G >= f.width)  // the last atom's groups past the row
      for (int e = g + 1; (e & 3) != 0; ++e) f.hsf[fp4::scale_offset(t, e, atoms)] = static_cast<uint8_t>(fp4::F4<FMT>::kScaleFill);
  }
}

template <typename TS, typename TB, int VEC, int I>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormFwd f, int row_ctas) {
  __shared__ float2 red[2][32];
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) >= row_ctas) {
    // the scale atoms' rows past the last token, a word (4 groups) per thread
    const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width);
    const int pad = static_cast<int>((128 - (f.tokens & 127)) & 127);
    const int64_t i = (blockIdx.x - row_ctas) * static_cast<int64_t>(blockDim.x * blockDim.y) + threadIdx.y * blockDim.x + threadIdx.x;
    if (i < pad * atoms)
      *reinterpret_cast<uint32_t*>(f.hsf + fp4::scale_offset(f.tokens + i / atoms, i % atoms * 4, atoms)) = f.h_fmt == 0 ? 0u : 0x7F7F7F7Fu;
    return;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= f.tokens) return;  // (a row of one warp: no barrier follows)
  int turn = 0;
  const int D = static_cast<int>(f.width), step = blockDim.x * VEC, c0 = threadIdx.x * VEC;
  const float alpha = f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f;
  const TS* r = static_cast<const TS*>(f.r) + t * f.ld_r;
  float x[I][VEC], n[I][VEC];
#pragma unroll
  for (int i = 0; i < I; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[i][j] = n[i][j] = 0.0f;
    if (c0 + i * step < D) load_stream<VEC>(r + c0 + i * step, x[i]);
  }
  if (f.o != nullptr) {
    const TB* o = static_cast<const TB*>(f.o) + t * f.ld_o;
    const TB* gate = f.gate != nullptr ? static_cast<const TB*>(f.gate) + t / f.gate_rows * f.ld_gate : nullptr;
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (c0 + i * step < D) load_stream<VEC>(o + c0 + i * step, n[i]);
    const float2 post = held_stat<VEC, I>(f.post, D, f.eps, n, red, turn);
    if (threadIdx.x == 0 && f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = post;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = c0 + i * step;
      if (c >= D) break;
      float w[VEC], b[VEC], g[VEC];
      if (f.w_post != nullptr) load_param<VEC>(f.w_post + c, w);
      if (f.b_post != nullptr) load_param<VEC>(f.b_post + c, b);
      if (gate != nullptr) load_param<VEC>(gate + c, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float z = (n[i][j] - post.x) * post.y;
        if (f.w_post != nullptr) z *= w[j];
        if (f.b_post != nullptr) z += b[j];
        const float v = x[i][j] * alpha;
        x[i][j] = gate != nullptr ? fmaf(g[j], z, v) : v + z;
      }
    }
  } else {
    if (threadIdx.x == 0 && f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = make_float2(0.0f, 1.0f);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] *= alpha;
  }
  if (f.r_out != nullptr) {  // (r may be r_out: every thread has read what it writes)
    TS* out = static_cast<TS*>(f.r_out) + t * f.ld_r_out;
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (c0 + i * step < D) store_stream<VEC>(out + c0 + i * step, x[i]);
  }
  const float2 pre = held_stat<VEC, I>(f.pre, D, f.eps, x, red, turn);
  if (threadIdx.x == 0 && f.stat_pre != nullptr) reinterpret_cast<float2*>(f.stat_pre)[t] = pre;
  if (f.h == nullptr && f.hq == nullptr) return;
  TB* h = static_cast<TB*>(f.h) + t * f.ld_h;
  const float hs = f.hq != nullptr && f.h_scale != nullptr ? __ldg(f.h_scale) : 1.0f;
  const int64_t atoms = fp4::atoms_along(f.h_fmt, D), pitch = fp4::row_bytes(D);
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = c0 + i * step;
    if (c >= D) break;
    float w[VEC], b[VEC], y[VEC];
    if (f.w_pre != nullptr) load_param<VEC>(f.w_pre + c, w);
    if (f.b_pre != nullptr) load_param<VEC>(f.b_pre + c, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      y[j] = (x[i][j] - pre.x) * pre.y;
      if (f.w_pre != nullptr) y[j] *= w[j];
      if (f.b_pre != nullptr) y[j] += b[j];
    }
    if (f.h != nullptr) store_stream<VEC>(h + c, y);
    if (f.hq != nullptr) {
      if (f.h_fmt == 0)
        emit_codes<0, VEC>(f, y, t, c, hs, pitch, atoms);
      else
        emit_codes<1, VEC>(f, y, t, c, hs, pitch, atoms);
    }
  }
}

template <typename TS, typename TB, int VEC, int I>
cudaError_t launch_rows(const NormFwd& f, cudaStream_t stream) {
  const int warps = static_cast<int>((f.width + 32 * VEC * I - 1) / (32 * VEC * I));
  const int rows = warps == 1 ? 4 : 1;
  const int64_t row_ctas = (f.tokens + rows - 1) / rows;
  int64_t fill = 0;
  if (f.hq != nullptr) {
    const int64_t words = ((128 - (f.tokens & 127)) & 127) * fp4::atoms_along(f.h_fmt, f.width);
    fill = (words + 32 * warps * rows - 1) / (32 * warps * rows);
  }
  return launch_pdl(norm_fwd_kernel<TS, TB, VEC, I>, dim3(static_cast<unsigned>(row_ctas + fill)), dim3(32 * warps, rows), 0, stream, f,
                    static_cast<int>(row_ctas));
}

template <typename TS, typename TB>
cudaError_t fwd_as(const NormFwd& f, cudaStream_t stream) {
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  const bool vec = f.width % 4 == 0 && rows_aligned(f.r, f.ld_r, ss, 4 * ss) && rows_aligned(f.r_out, f.ld_r_out, ss, 4 * ss) &&
                   rows_aligned(f.o, f.ld_o, bs, 4 * bs) && rows_aligned(f.h, f.ld_h, bs, 4 * bs) && rows_aligned(f.gate, f.ld_gate, bs, 4 * bs) &&
                   rows_aligned(f.w_post, 0, 4, 16) && rows_aligned(f.b_post, 0, 4, 16) && rows_aligned(f.w_pre, 0, 4, 16) && rows_aligned(f.b_pre, 0, 4, 16);
  // 32 elements per lane keep enough loads in flight for the memory's rate; with no more rows than a few per
  // SM the latency counts instead, and a row is spread over four times the lanes
  const bool few = f.tokens <= 2ll * num_sms();
  if (f.width <= 256 || (few && f.width <= 4096)) return vec ? launch_rows<TS, TB, 4, 2>(f, stream) : launch_rows<TS, TB, 1, 8>(f, stream);
  if (f.width <= 16384) return vec ? launch_rows<TS, TB, 4, 8>(f, stream) : launch_rows<TS, TB, 1, 32>(f, stream);
  const int64_t most = 8ll * num_sms();
  return launch_pdl(norm_fwd_any_kernel<TS, TB>, dim3(static_cast<unsigned>(f.tokens < most ? f.tokens : most)), dim3(kThreads), 0, stream, f);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& f, cudaStream_t stream) {
  if (f.stream_f32)
    return f.block_f32 ? fwd_as<float, float>(f, stream) : fwd_as<float, bf16>(f, stream);
  return f.block_f32 ? fwd_as<bf16, float>(f, stream) : fwd_as<bf16, bf16>(f, stream);
}

}  // namespace fp8gb
