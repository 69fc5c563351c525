// qk_rope.cu -- heads of queries and keys: norm over each head and rotation by the token's position, forward and
// backward (mathematics and layout: heads.cuh).
//
// What bounds it: memory. Forward reads and writes each element once; backward reads the gradient and, with a norm, the
// input, and writes one gradient. A token's angles are worked out once per item (a token and a run of its heads)
// and serve all its rows; a lane's norm weight, angle and amplitude are one factor per member of a pair
//   y_u = r (u uc - v vs),  y_v = r (u us + v vc),   uc = w_u cos a, us = w_u sin a, vs = w_v sin a, vc = w_v cos a,
// and the arithmetic works on two pairs at once (fp32x2). Measured, 16384 tokens of 32 + 8 heads of 128 in bf16 with norms: forward 52.8 us,
// 6.35 TB/s (0.94 of a copy; 54.0 on another box); backward 96 us, 5.2 TB/s, some 4 of them the sum of the weights' gradients: rows in registers are what it
// has too few of on their way.
// Backward: with (du, dv) the incoming pair turned back, z = x r, dz = w d:
//   dx = r (dz - z mean(dz z)),   dw = sum over tokens and heads of d z.
#include "heads.cuh"

namespace fp8gb {
namespace {

using namespace heads;

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Of the forward: small CTAs, a warp's slot is free again when its CTA's last warp is done (16384 tokens of 40 heads of 128: 52.8 us;
// CTAs of 128 threads 53.3, of 256 54.6).
constexpr int kFwdThreads = 64, kFwdWarps = kFwdThreads / 32;

struct Args {
  Turn t;
  Heads part[2];
  TurnGrad grad[2];
  int per;            // heads of one item
  int items0, items1; // items of a token: of the queries, of the keys
  int64_t total0, total;  // items of all queries, in all
  float* sums;        // [CTAs, 2, head_dim]
};

template <typename T>
__device__ __forceinline__ const T* row_of(const void* p, int64_t ld, int64_t hs, int64_t t, int h) {
  return static_cast<const T*>(p) + t * ld + h * hs;
}

// Item i: a token, a part, and heads h0 .. h1 - 1 of it. All tokens' queries come before the keys: a kernel that steps through the
// items takes the same share of the long and of the short ones with every warp.
struct Item {
  int64_t token;
  int part, h0, h1;
};
__device__ __forceinline__ Item item_of(int64_t i, const Args& g) {
  Item m;
  m.part = i >= g.total0;
  if (m.part) i -= g.total0;
  const int items = m.part ? g.items1 : g.items0;
  m.token = items == 1 ? i : i >> 32 == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(items) : i / items;
  m.h0 = static_cast<int>(i - m.token * items) * g.per;
  m.h1 = min(m.h0 + g.per, g.part[m.part].n);
  return m;
}

// CTAs of the backward on an SM: with registers for two turns of two rows each (with a norm; 16384 tokens of 40 heads of 128: 95 us; a row a
// turn with 3 CTAs 106, two rows 124, three rows 106, four 99; with the next item's rows fetched into L2 by bulk prefetches
// 111, or loaded before an item ends 95).
constexpr int kBwdCtas = 2;

// Rows of a turn, so that the next turn's loads fit beside them.
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 4 : 2;

template <typename T, bool INTER, int LPR, bool NORM, bool PARTIAL>
__global__ void __launch_bounds__(kFwdThreads, 12) qk_rope_fwd_kernel(const __grid_constant__ Args g) {
  constexpr int RPW = 32 / LPR, U = kRows<T>;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const Lane a = lane_of<INTER>(lane % LPR, g.t.head_dim, g.t.rot_dims);
  pdl_wait();
  pdl_trigger();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kFwdWarps + (threadIdx.x >> 5);
  if (i >= g.total) return;
  const Item m = item_of(i, g);
  const Heads& p = g.part[m.part];
  const T* in = row_of<T>(p.in, p.ld_in, p.hs_in, m.token, 0);
  T* out = static_cast<T*>(p.out) + m.token * p.ld_out;
  // (lanes past the head hold zeros; a row past the last one is the last one again, and not stored)
  Raw<T, INTER> raw[U], next[U] = {};
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (a.in) next[j].load(in + min(h0 + j * RPW + sub, m.h1 - 1) * p.hs_in, a.o0, a.o1);
  };
  load(m.h0);
  float c[4], s[4], wu[4], wv[4];
  angles<LPR>(a, g.t.turns, g.t.rot_dims, g.t.pos != nullptr ? __ldg(g.t.pos + m.token) : static_cast<int32_t>(m.token), g.t.amplitude, c, s);
  weights<INTER>(a, p.w, wu, wv);
  const Factors f = factors(c, s, wu, wv);
  const float inv_dim = 1.0f / static_cast<float>(g.t.head_dim);
#pragma unroll 1
  for (int h0 = m.h0; h0 < m.h1; h0 += U * RPW) {
#pragma unroll
    for (int j = 0; j < U; ++j) raw[j] = next[j];
    if (h0 + U * RPW < m.h1) load(h0 + U * RPW);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      Pair u[2], v[2], yu[2], yv[2];
      raw[j].get(u, v);
      turn<LPR, NORM, INTER, PARTIAL>(a, f, inv_dim, g.t.eps, u, v, yu, yv);
      const int h = h0 + j * RPW + sub;
      if (a.in && h < m.h1) Raw<T, INTER>::put(out + h * p.hs_out, a.o0, a.o1, yu, yv);
    }
  }
}

template <typename T, bool INTER, int LPR, bool NORM, bool DW, bool PARTIAL>
__global__ void __launch_bounds__(kThreads, kBwdCtas) qk_rope_bwd_kernel(const __grid_constant__ Args g) {
  constexpr int RPW = 32 / LPR, U = NORM ? 2 : kRows<T>;
  // sums for dw: a warp's columns of both parts, added to after each item
  __shared__ float share[DW ? kWarps : 1][2][DW ? LPR * 8 : 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
  const Lane a = lane_of<INTER>(lane % LPR, g.t.head_dim, g.t.rot_dims);
  const float inv_dim = 1.0f / static_cast<float>(g.t.head_dim);
  auto column = [&](int k, int member) { return INTER ? a.o0 + 2 * k + member : (member == 0 ? a.o0 : a.o1) + k; };
  if constexpr (DW) {
    for (int x = lane; x < 2 * LPR * 8; x += 32) share[warp][x / (LPR * 8)][x % (LPR * 8)] = 0.0f;
    __syncwarp();
  }
  pdl_wait();
  pdl_trigger();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < g.total; i += step) {
    const Item m = item_of(i, g);
    const Heads& p = g.part[m.part];
    const TurnGrad& b = g.grad[m.part];
    const T* dy = row_of<T>(b.dy, b.ld_dy, b.hs_dy, m.token, 0);
    const T* in = NORM ? row_of<T>(p.in, p.ld_in, p.hs_in, m.token, 0) : nullptr;
    T* dx = static_cast<T*>(b.dx) + m.token * b.ld_dx;
    Raw<T, INTER> rd[U], rx[U], next_d[U] = {}, next_x[U] = {};
    auto load = [&](int h0) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = min(h0 + j * RPW + sub, m.h1 - 1);
        if (a.in) {
          next_d[j].load(dy + h * b.hs_dy, a.o0, a.o1);
          if constexpr (NORM) next_x[j].load(in + h * p.hs_in, a.o0, a.o1);
        }
      }
    };
    load(m.h0);
    float c[4], s[4], wu[4], wv[4];
    angles<LPR>(a, g.t.turns, g.t.rot_dims, g.t.pos != nullptr ? __ldg(g.t.pos + m.token) : static_cast<int32_t>(m.token), g.t.amplitude, c, s);
    if constexpr (NORM) weights<INTER>(a, p.w, wu, wv);
    Pair au[2] = {}, av[2] = {}, pc[2], ps[2], ns[2], pu[2], pv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      pc[k] = pair(c[2 * k], c[2 * k + 1]);
      ps[k] = pair(s[2 * k], s[2 * k + 1]);
      ns[k] = pair(-s[2 * k], -s[2 * k + 1]);
      if constexpr (NORM) pu[k] = pair(wu[2 * k], wu[2 * k + 1]), pv[k] = pair(wv[2 * k], wv[2 * k + 1]);
    }
#pragma unroll 1
    for (int h0 = m.h0; h0 < m.h1; h0 += U * RPW) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        rd[j] = next_d[j];
        if constexpr (NORM) rx[j] = next_x[j];
      }
      if (h0 + U * RPW < m.h1) load(h0 + U * RPW);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        Pair du[2], dv[2], yu[2], yv[2];
        const int h = h0 + j * RPW + sub;
        const bool live = a.in && h < m.h1;
        rd[j].get(du, dv);
        Pair tu[2], tv[2];
        turning<INTER, PARTIAL>(a.turned, 0.0f, du, tu);   // (times -sin)
        turning<INTER, PARTIAL>(a.turned, -0.0f, dv, tv);  // (times sin)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          yu[k] = fma2(du[k], pc[k], mul2(tv[k], ps[k]));
          yv[k] = fma2(dv[k], pc[k], mul2(tu[k], ns[k]));
        }
        if constexpr (NORM) {
          Pair u[2], v[2];
          rx[j].get(u, v);
#pragma unroll
          for (int k = 0; k < 2; ++k) tu[k] = mul2(yu[k], pu[k]), tv[k] = mul2(yv[k], pv[k]);
          float q = sum2(fma2(u[0], u[0], fma2(u[1], u[1], fma2(v[0], v[0], mul2(v[1], v[1])))));
          float e = sum2(fma2(u[0], tu[0], fma2(u[1], tu[1], fma2(v[0], tv[0], mul2(v[1], tv[1])))));
#pragma unroll
          for (int x = LPR / 2; x > 0; x >>= 1) {
            q += __shfl_xor_sync(0xFFFFFFFFu, q, x);
            e += __shfl_xor_sync(0xFFFFFFFFu, e, x);
          }
          // dx = r (t - z mean(t z)) with z = x r first: r^3 leaves fp32's range where rows are beyond 10^13 or below 10^-13
          const float r = rsqrtf(fmaf(q, inv_dim, g.t.eps));
          const Pair rr = both(r), m = both(-(e * r) * inv_dim);
#pragma unroll
          for (int k = 0; k < 2; ++k) u[k] = mul2(u[k], rr), v[k] = mul2(v[k], rr);
          if constexpr (DW) {
            if (live) {  // (not a factor of 0 for the others: they repeat the last row, and an infinity of it times 0 is no 0)
#pragma unroll
              for (int k = 0; k < 2; ++k) au[k] = fma2(yu[k], u[k], au[k]), av[k] = fma2(yv[k], v[k], av[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            yu[k] = mul2(fma2(u[k], m, tu[k]), rr);
            yv[k] = mul2(fma2(v[k], m, tv[k]), rr);
          }
        }
        if (live && b.dx != nullptr) Raw<T, INTER>::put(dx + h * b.hs_dx, a.o0, a.o1, yu, yv);
      }
    }
    if constexpr (DW) {
      const float2 pairs[4] = {split(au[0]), split(au[1]), split(av[0]), split(av[1])};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float x = k & 1 ? pairs[k >> 1].y : pairs[k >> 1].x;
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        if (sub == 0 && a.in) share[warp][m.part][column(k & 3, k >> 2)] += x;
      }
    }
  }
  if constexpr (DW) {
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * g.t.head_dim; x += kThreads) {
      const int p = x / g.t.head_dim, d = x - p * g.t.head_dim;
      float q = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) q += share[w][p][d];
      g.sums[static_cast<int64_t>(blockIdx.x) * 2 * g.t.head_dim + x] = q;
    }
  }
}

// Rows of single elements, a warp each; forward (BWD false) or backward. (8192 tokens of 40 heads of 128 in bf16 with norms, 60 elements turning: 104 us
// with 4 CTAs an SM, 114 with 3; backward 277.)
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 4) qk_rope_any_kernel(const __grid_constant__ Args g) {
  __shared__ float share[kWarps][256];
  __shared__ float sums[kWarps][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = g.t.head_dim, R = g.t.rot_dims;
  const float inv_dim = 1.0f / static_cast<float>(D);
  float acc[2][8] = {};
  pdl_wait();
  pdl_trigger();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < g.total; i += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Item m = item_of(i, g);
    const Heads& p = g.part[m.part];
    const TurnGrad& b = g.grad[m.part];
    const int32_t pos = g.t.pos != nullptr ? __ldg(g.t.pos + m.token) : static_cast<int32_t>(m.token);
    // of element d: its partner, and cos, +-sin with which y_d = x_d c + x_partner s (backward: the other sign)
    float c[8], s[8], w[8];
    int mate[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int d = lane + 32 * k;
      c[k] = 1.0f, s[k] = 0.0f, w[k] = 1.0f, mate[k] = d & 255;
      if (d < R) {
        const bool second = g.t.interleaved ? d & 1 : d >= R / 2;
        const int pair = g.t.interleaved ? d >> 1 : second ? d - R / 2 : d;
        const float2 t = cos_sin(__ldg(g.t.turns + pair), pos);
        c[k] = t.x * g.t.amplitude;
        s[k] = t.y * g.t.amplitude * (second != BWD ? 1.0f : -1.0f);
        mate[k] = g.t.interleaved ? d ^ 1 : second ? d - R / 2 : d + R / 2;
      }
      if (d < D && p.w != nullptr) w[k] = __ldg(p.w + d);
    }
    for (int h = m.h0; h < m.h1; ++h) {
      float x[8], r = 1.0f;
      const T* in = row_of<T>(p.in, p.ld_in, p.hs_in, m.token, h);
      const T* dy = row_of<T>(b.dy, b.ld_dy, b.hs_dy, m.token, h);
      const bool reads_x = !BWD || g.t.norm;
      float q = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = lane + 32 * k;
        x[k] = reads_x && d < D ? element(in + d) : 0.0f;
        q = fmaf(x[k], x[k], q);
      }
      if (g.t.norm) r = rsqrtf(fmaf(row_sum<32>(q), inv_dim, g.t.eps));
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = lane + 32 * k;
        y[k] = BWD ? (d < D ? element(dy + d) : 0.0f) : x[k] * r * w[k];
        share[warp][d] = y[k];
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float t = fmaf(y[k], c[k], share[warp][mate[k]] * s[k]);
        y[k] = lane + 32 * k < R ? t : y[k];  // (the others stay: 0 times an infinity is no 0)
      }
      __syncwarp();
      if constexpr (BWD) {
        if (g.t.norm) {
          float e = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float z = x[k] * r;
            if (m.part == 0)
              acc[0][k] = fmaf(y[k], z, acc[0][k]);
            else
              acc[1][k] = fmaf(y[k], z, acc[1][k]);
            e = fmaf(y[k] * w[k], z, e);
          }
          e = row_sum<32>(e) * inv_dim;
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = r * (y[k] * w[k] - x[k] * r * e);
        }
      }
      T* out = BWD ? static_cast<T*>(b.dx) : static_cast<T*>(p.out);
      const int64_t at = BWD ? m.token * b.ld_dx + h * b.hs_dx : m.token * p.ld_out + h * p.hs_out;
      if (out != nullptr)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (lane + 32 * k < D) set_element(out + at + lane + 32 * k, y[k]);
    }
  }
  if (BWD && g.sums != nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[warp][0][lane + 32 * k] = acc[0][k], sums[warp][1][lane + 32 * k] = acc[1][k];
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
      const int part = x / D, d = x - part * D;
      float q = 0.0f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) q += sums[j][part][d];
      g.sums[static_cast<int64_t>(blockIdx.x) * 2 * D + x] = q;
    }
  }
}

// dw of both parts from the CTAs' sums: a CTA for 32 columns, a warp for every 32nd CTA's sums (8 loads on their way at a time), then
// the warps' in order.
__global__ void __launch_bounds__(1024) qk_rope_dw_kernel(const float* sums, int ctas, int dim, float* dw_q, float* dw_k) {
  __shared__ float share[32][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x = blockIdx.x * 32 + lane;
  float q = 0.0f;
#pragma unroll 8
  for (int c = warp; c < ctas; c += 32) q += x < 2 * dim ? __ldcg(sums + static_cast<int64_t>(c) * 2 * dim + x) : 0.0f;
  share[warp][lane] = q;
  __syncthreads();
  if (warp > 0 || x >= 2 * dim) return;
  float* out = x < dim ? dw_q : dw_k;
  if (out == nullptr) return;
  q = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) q += share[w][lane];
  out[x < dim ? x : x - dim] = q;
}

int bwd_ctas() { return kBwdCtas * num_sms(); }

bool chunks_of(const void* p, int64_t ld, int64_t hs, int64_t bytes, int64_t elem) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * elem % bytes == 0 && hs * elem % bytes == 0);
}

template <typename F>
cudaError_t by_kind(const Turn& t, F&& f) {
  const int lpr = t.head_dim <= 64 ? 8 : t.head_dim <= 128 ? 16 : 32;
#define FP8GB_LPR(T, I) (lpr == 8 ? f.template operator()<T, I, 8>() : lpr == 16 ? f.template operator()<T, I, 16>() : f.template operator()<T, I, 32>())
  if (t.f32) return t.interleaved ? FP8GB_LPR(float, true) : FP8GB_LPR(float, false);
  return t.interleaved ? FP8GB_LPR(bf16, true) : FP8GB_LPR(bf16, false);
#undef FP8GB_LPR
}

// Items: a token's heads in runs of `per`, so that there are at least `want` of them where that leaves a run at least `least` heads.
void set_items(Args& g, int64_t want, int least) {
  const int heads = max(g.part[0].n, g.part[1].n);
  const int64_t runs = min(static_cast<int64_t>((heads + least - 1) / least), max(int64_t{1}, (want + g.t.tokens - 1) / g.t.tokens));
  g.per = static_cast<int>((heads + runs - 1) / runs);
  g.items0 = (g.part[0].n + g.per - 1) / g.per;
  g.items1 = (g.part[1].n + g.per - 1) / g.per;
  g.total0 = g.t.tokens * g.items0;
  g.total = g.total0 + g.t.tokens * g.items1;
}

// Heads that turn in part have kernels of their own.
template <typename T, bool I, int L, bool NORM>
auto fwd_kernel(bool partial) {
  return partial ? qk_rope_fwd_kernel<T, I, L, NORM, true> : qk_rope_fwd_kernel<T, I, L, NORM, false>;
}
template <typename T, bool I, int L, bool NORM, bool DW>
auto bwd_kernel(bool partial) {
  return partial ? qk_rope_bwd_kernel<T, I, L, NORM, DW, true> : qk_rope_bwd_kernel<T, I, L, NORM, DW, false>;
}

struct FwdLaunch {
  const Args& g;
  cudaStream_t s;
  template <typename T, bool I, int L>
  cudaError_t operator()() const {
    const bool partial = g.t.rot_dims < g.t.head_dim;
    return launch_pdl(g.t.norm ? fwd_kernel<T, I, L, true>(partial) : fwd_kernel<T, I, L, false>(partial), dim3(static_cast<unsigned>((g.total + kFwdWarps - 1) / kFwdWarps)), dim3(kFwdThreads), 0, s, g);
  }
};

struct BwdLaunch {
  const Args& g;
  cudaStream_t s;
  int ctas;
  template <typename T, bool I, int L>
  cudaError_t operator()() const {
    const bool partial = g.t.rot_dims < g.t.head_dim;
    auto* k = g.t.norm ? (g.sums != nullptr ? bwd_kernel<T, I, L, true, true>(partial) : bwd_kernel<T, I, L, true, false>(partial)) : bwd_kernel<T, I, L, false, false>(partial);
    return launch_pdl(k, dim3(ctas), dim3(kThreads), 0, s, g);
  }
};

}  // namespace

cudaError_t launch_qk_rope_fwd(const Turn& f, const Heads (&part)[2], cudaStream_t stream) {
  Args g{};
  g.t = f;
  g.part[0] = part[0];
  g.part[1] = part[1];
  const int64_t elem = f.f32 ? 4 : 2, bytes = f.f32 || f.interleaved ? 16 : 8;
  bool vec = f.head_dim % 8 == 0 && (f.interleaved || f.rot_dims % 8 == 0);
  for (const Heads& p : part)
    if (p.n > 0) vec = vec && chunks_of(p.in, p.ld_in, p.hs_in, bytes, elem) && chunks_of(p.out, p.ld_out, p.hs_out, bytes, elem);
  set_items(g, int64_t{64} * num_sms(), 8);
  if (vec) return by_kind(f, FwdLaunch{g, stream});
  const unsigned ctas = static_cast<unsigned>(min((g.total + kWarps - 1) / kWarps, int64_t{8} * num_sms()));
  return f.f32 ? launch_pdl(qk_rope_any_kernel<float, false>, dim3(ctas), dim3(kThreads), 0, stream, g)
               : launch_pdl(qk_rope_any_kernel<bf16, false>, dim3(ctas), dim3(kThreads), 0, stream, g);
}

int64_t qk_rope_bwd_workspace_bytes(const Turn& f) { return static_cast<int64_t>(bwd_ctas()) * 2 * f.head_dim * 4; }

cudaError_t launch_qk_rope_bwd(const Turn& f, const Heads (&part)[2], const TurnGrad (&grad)[2], void* ws, cudaStream_t stream) {
  Args g{};
  g.t = f;
  bool vec = f.head_dim % 8 == 0 && (f.interleaved || f.rot_dims % 8 == 0);
  const int64_t elem = f.f32 ? 4 : 2, bytes = f.f32 || f.interleaved ? 16 : 8;
  for (int p = 0; p < 2; ++p) {
    g.part[p] = part[p];
    g.grad[p] = grad[p];
    if (part[p].n == 0) continue;
    vec = vec && chunks_of(grad[p].dy, grad[p].ld_dy, grad[p].hs_dy, bytes, elem) && chunks_of(grad[p].dx, grad[p].ld_dx, grad[p].hs_dx, bytes, elem) &&
          (!f.norm || chunks_of(part[p].in, part[p].ld_in, part[p].hs_in, bytes, elem));
  }
  const bool dw = grad[0].dw != nullptr || grad[1].dw != nullptr;
  if (dw) g.sums = static_cast<float*>(ws);
  set_items(g, int64_t{4} * bwd_ctas() * kWarps, 8);
  const int ctas = static_cast<int>(min((g.total + kWarps - 1) / kWarps, static_cast<int64_t>(bwd_ctas())));
  cudaError_t e;
  if (vec)
    e = by_kind(f, BwdLaunch{g, stream, ctas});
  else
    e = f.f32 ? launch_pdl(qk_rope_any_kernel<float, true>, dim3(ctas), dim3(kThreads), 0, stream, g)
              : launch_pdl(qk_rope_any_kernel<bf16, true>, dim3(ctas), dim3(kThreads), 0, stream, g);
  if (e != cudaSuccess || !dw) return e;
  const float* sums = g.sums;
  return launch_pdl(qk_rope_dw_kernel, dim3((2 * f.head_dim + 31) / 32), dim3(1024), 0, stream, sums, ctas, f.head_dim, grad[0].dw, grad[1].dw);
}

}  // namespace fp8gb
