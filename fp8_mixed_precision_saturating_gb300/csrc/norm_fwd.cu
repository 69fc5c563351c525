// norm_fwd.cu -- forward of the norms around a block with its gate and the residual's scale (HBM-bound).
#include "norm_emit.cuh"

namespace fp8gb {
namespace {

using namespace norms;

// Mean and 1 / root of a row whose element c is value(c).
template <typename F>
__device__ __forceinline__ float2 row_stat(int kind, int64_t width, float eps, Red& red, int& turn, F value) {
  float2 st = make_float2(0.0f, 1.0f);
  if (kind == kNone) return st;
  const float inv = 1.0f / static_cast<float>(width);
  if (kind == kLayer) {
    float a = 0.0f;
    for (int64_t c = threadIdx.x; c < width; c += kThreads) a += value(c);
    st.x = cta_sum(a, red, turn) * inv;
  }
  float a = 0.0f;
  for (int64_t c = threadIdx.x; c < width; c += kThreads) {
    const float z = value(c) - st.x;
    a = fmaf(z, z, a);
  }
  st.y = inv_sqrt(fmaf(cta_sum(a, red, turn), inv, eps));
  return st;
}

// Any width and alignment: one CTA per token, the row read again for every pass over it. 2048 x 20480 bf16 252 us, where
// the rows' bytes take 49.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) norm_fwd_any_kernel(const NormFwd f) {
  __shared__ Red red;
  int turn = 0;
  red.clear();
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
      const uint32_t least = fp4::least_scale(s);
      const int64_t atoms = fp4::atoms_along(f.h_fmt, f.width), pitch = fp4::row_bytes(f.width);
      const int group = f.h_fmt == 0 ? 16 : 32;
      for (int64_t g = threadIdx.x; g < f.width / group; g += kThreads) {
        uint32_t a = 0;
        auto hv = [&](int64_t c) { return affine((mid(c) - pre.x) * pre.y, f.w_pre, f.b_pre, c); };
        for (int i = 0; i < group; ++i) a = max(a, __float_as_uint(hv(g * group + i)) & 0x7FFFFFFFu);
        float mul;
        const uint32_t b = f.h_fmt == 0 ? fp4::group_scale<0>(a, s, least, mul) : fp4::group_scale<1>(a, s, least, mul);
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
// The row's elements are read once and stay in registers through both statistics; the parameters come from L1,
// where the streamed rows do not displace them. `blockDim.x / 32` warps share a row; a warp that holds a whole row
// needs no barrier, and blockDim.y such rows share a CTA.
template <int VEC, int E, bool FULL>
__device__ __forceinline__ float2 held_stat(int kind, int width, float eps, const Pair (&v)[E / 2], int left, Red& red, int& turn) {
  float2 st = make_float2(0.0f, 1.0f);
  if (kind == kNone) return st;
  const float inv = 1.0f / static_cast<float>(width);
  Pair q = both(0.0f);
  if (kind == kLayer) {
    Pair a = both(0.0f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) a = add2(a, v[i]);  // (zero past the row)
    st.x = cta_sum(sum2(a), red, turn) * inv;
    const Pair m = both(-st.x);
    Pair z[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) z[i] = add2(v[i], m);
    Row<VEC, E, FULL>::clear(z, left);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) q = fma2(z[i], z[i], q);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) q = fma2(v[i], v[i], q);
  }
  st.y = inv_sqrt(fmaf(cta_sum(sum2(q), red, turn), inv, eps));
  return st;
}

// x <- ((x - mean) rstd) w + b, the mean taken off before the scaling so that a large one does not cancel
template <int VEC, int E, bool FULL>
__device__ __forceinline__ void held_affine(Pair (&x)[E / 2], int kind, float2 st, const float* w, const float* b, int c, int left) {
  if (kind == kNone) return;
  const Pair rstd = both(st.y);
  if (kind == kLayer) {
    const Pair m = both(-st.x);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(add2(x[i], m), rstd);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], rstd);
  }
  if (w != nullptr) {
    Pair p[E / 2];
    Row<VEC, E, FULL>::template load<false>(w + c, left, p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], p[i]);
  }
  if (b != nullptr) {
    Pair p[E / 2];
    Row<VEC, E, FULL>::template load<false>(b + c, left, p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = add2(x[i], p[i]);
  }
}

// A row per CTA (or per warp), loaded straight into registers.
template <typename TS, typename TB, int VEC, int E, bool FULL>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormFwd f, int row_ctas, uint32_t gate_rows) {
  using R = Row<VEC, E, FULL>;
  __shared__ Red red;
  __shared__ float table[4][8];
  if (blockDim.x > 32) red.clear();
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) >= row_ctas) {
    const int64_t threads = static_cast<int64_t>(blockDim.x) * blockDim.y;
    fill_scales(f, (blockIdx.x - row_ctas) * threads + threadIdx.y * blockDim.x + threadIdx.x, (gridDim.x - row_ctas) * threads);
    return;
  }
  const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= f.tokens) return;  // (a row of one warp: no barrier follows)
  int turn = 0;
  const int c = R::first(threadIdx.x >> 5, threadIdx.x & 31), left = static_cast<int>(f.width) - c;
  Pair x[E / 2], n[E / 2];
  R::template load<true>(static_cast<const TS*>(f.r) + t * f.ld_r + c, left, x);
  if (f.o != nullptr) R::template load<true>(static_cast<const TB*>(f.o) + t * f.ld_o + c, left, n);
  const float alpha = f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f;
  fill_table(f, table[threadIdx.y], threadIdx.x);
  const int D = static_cast<int>(f.width);
  if (f.o != nullptr) {
    const float2 post = held_stat<VEC, E, FULL>(f.post, D, f.eps, n, left, red, turn);
    if (threadIdx.x == 0 && f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = post;
    held_affine<VEC, E, FULL>(n, f.post, post, f.w_post, f.b_post, c, left);
    const Pair a = both(alpha);
    if (f.gate != nullptr) {
      Pair g[E / 2];
      R::template load<false>(static_cast<const TB*>(f.gate) + (t / gate_rows) * f.ld_gate + c, left, g);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = fma2(g[i], n[i], mul2(x[i], a));
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = fma2(x[i], a, n[i]);
    }
  } else {
    if (threadIdx.x == 0 && f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = make_float2(0.0f, 1.0f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], both(alpha));
  }
  R::clear(x, left);  // (past the row: what the norm made of nothing)
  // (r may be r_out: every thread has read what it writes)
  if (f.r_out != nullptr) R::store(static_cast<TS*>(f.r_out) + t * f.ld_r_out + c, left, x);
  const float2 pre = held_stat<VEC, E, FULL>(f.pre, D, f.eps, x, left, red, turn);
  if (threadIdx.x == 0 && f.stat_pre != nullptr) reinterpret_cast<float2*>(f.stat_pre)[t] = pre;
  if (f.h == nullptr && f.hq == nullptr) return;
  held_affine<VEC, E, FULL>(x, f.pre, pre, f.w_pre, f.b_pre, c, left);
  if (f.h != nullptr) R::store(static_cast<TB*>(f.h) + t * f.ld_h + c, left, x);
  if (f.hq != nullptr) {
    if (blockDim.x > 32)
      __syncthreads();
    else
      __syncwarp();
    if (f.h_fmt == 0)
      emit_row<0, VEC, E>(f, x, t, c, left, table[threadIdx.y]);
    else
      emit_row<1, VEC, E>(f, x, t, c, left, nullptr);
  }
}

template <typename TS, typename TB, int VEC, int E, bool FULL>
cudaError_t launch_rows(const NormFwd& f, cudaStream_t stream) {
  const int warps = static_cast<int>((f.width + 32 * E - 1) / (32 * E));
  const int rows = warps == 1 ? 4 : 1;
  const int64_t row_ctas = (f.tokens + rows - 1) / rows;
  int64_t fill = 0;
  if (f.hq != nullptr) {
    const int64_t words = ((128 - (f.tokens & 127)) & 127) * fp4::atoms_along(f.h_fmt, f.width);
    fill = (words + 32 * warps * rows - 1) / (32 * warps * rows);
  }
  return launch_pdl(norm_fwd_kernel<TS, TB, VEC, E, FULL>, dim3(static_cast<unsigned>(row_ctas + fill)), dim3(32 * warps, rows), 0, stream, f,
                    static_cast<int>(row_ctas), gate_rows_of(f));
}

template <typename TS, typename TB>
cudaError_t fwd_as(const NormFwd& f, cudaStream_t stream) {
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  const bool vec = f.width % 4 == 0 && rows_aligned(f.r, f.tokens, f.ld_r, ss, 4 * ss) && rows_aligned(f.r_out, f.tokens, f.ld_r_out, ss, 4 * ss) &&
                   rows_aligned(f.o, f.tokens, f.ld_o, bs, 4 * bs) && rows_aligned(f.h, f.tokens, f.ld_h, bs, 4 * bs) && rows_aligned(f.gate, gate_groups(f), f.ld_gate, bs, 4 * bs) &&
                   rows_aligned(f.w_post, 1, 0, 4, 16) && rows_aligned(f.b_post, 1, 0, 4, 16) && rows_aligned(f.w_pre, 1, 0, 4, 16) && rows_aligned(f.b_pre, 1, 0, 4, 16);
  bool taken = false;
  const cudaError_t e = launch_norm_fwd_ring(f, stream, &taken);
  if (e != cudaSuccess || taken) return e;
  // 16 elements a lane keep the loads of a wide row in flight (304 x 4096 3.5 us, with 8 4.3) and make a row of up to 512 columns
  // one warp's, without a barrier (60000 x 512 44 us, with 8 63). With 8 a row in between has shorter chains (1 x 768 2.4 us,
  // with 16 2.8; 1000 x 768 3.1, 3.4), and one of 256 columns is a warp's as well
  if (f.width <= 256 || (f.width > 512 && f.width < 1024)) {
    if (!vec) return launch_rows<TS, TB, 1, 8, false>(f, stream);
    return f.width % 256 == 0 ? launch_rows<TS, TB, 4, 8, true>(f, stream) : launch_rows<TS, TB, 4, 8, false>(f, stream);
  }
  if (f.width <= 8192) {
    // single elements: 8 a lane keep 48 registers and twice the warps on an SM (4099 x 1537, fp32 stream: 26.5 -> 19.0 us);
    // a row of more than 16 warps takes 16 a lane
    if (!vec && f.width <= 4096) return launch_rows<TS, TB, 1, 8, false>(f, stream);
    if (!vec) return launch_rows<TS, TB, 1, 16, false>(f, stream);
    return f.width % 512 == 0 ? launch_rows<TS, TB, 4, 16, true>(f, stream) : launch_rows<TS, TB, 4, 16, false>(f, stream);
  }
  if (f.width <= 16384 && vec) return launch_rows<TS, TB, 4, 32, false>(f, stream);
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
