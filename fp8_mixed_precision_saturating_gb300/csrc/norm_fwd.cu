// norm_fwd.cu -- forward of the norms around a block with its gate and the residual's scale (HBM-bound).
#include "fp4.cuh"
#include "norm.cuh"

namespace fp8gb {
namespace {

using namespace norms;

constexpr int kMostTeams = 12;  // rows that a CTA works on at once

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

// Any width and alignment: one CTA per token, the row read again for every pass over it.
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

// The row's parameters: in global memory, or copied to shared memory by a CTA that works on many rows (SHARED; the
// addresses, 0 for what is not there; the gate's row too where all tokens share it).
struct Shared {
  uint32_t w_post, b_post, w_pre, b_pre, gate;
};

template <bool SHARED, int VEC, int E, bool FULL>
__device__ __forceinline__ void param(const float* p, uint32_t at, int c, int left, Pair (&x)[E / 2]) {
  if constexpr (SHARED)
    Row<VEC, E, FULL>::load_shared(at, c, left, x);
  else
    Row<VEC, E, FULL>::template load<false>(p + c, left, x);
}

// x <- ((x - mean) rstd) w + b, the mean taken off before the scaling so that a large one does not cancel
template <bool SHARED, int VEC, int E, bool FULL>
__device__ __forceinline__ void held_affine(Pair (&x)[E / 2], int kind, float2 st, const float* w, uint32_t w_at, const float* b, uint32_t b_at, int c, int left) {
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
    param<SHARED, VEC, E, FULL>(w, w_at, c, left, p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], p[i]);
  }
  if (b != nullptr) {
    Pair p[E / 2];
    param<SHARED, VEC, E, FULL>(b, b_at, c, left, p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = add2(x[i], p[i]);
  }
}

// VEC consecutive elements of h as 4-bit codes, with their group's scale (16 or 32 neighbouring elements, held by
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
  float w[8] = {};
#pragma unroll
  for (int j = 0; j < VEC; ++j) w[j] = __fmul_rn(h[j], mul);
  uint32_t codes = fp4::cvt8_e2m1(w);
  if (b == fp4::F4<FMT>::kScaleNaN) codes = 0;
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

template <int FMT, int VEC, int E>
__device__ __forceinline__ void emit_row(const NormFwd& f, const Pair (&h)[E / 2], int64_t t, int c, int left) {
  const float s = f.h_scale != nullptr ? __ldg(f.h_scale) : 1.0f;
  const int64_t atoms = fp4::atoms_along(FMT, f.width), pitch = fp4::row_bytes(f.width);
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
      emit_codes<FMT, VEC>(f, v, t, c + 32 * VEC * i, s, pitch, atoms);
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

// x: a token's row of the stream, n: of the block's output (where there is one), both becoming what is made of them.
// `read` runs behind a barrier that all threads pass after they have read the row (RING: its place is free then).
template <typename TS, typename TB, int VEC, int E, bool FULL, bool RING, typename Read>
__device__ __forceinline__ bool one_row(const NormFwd& f, const Shared& par, Pair (&x)[E / 2], Pair (&n)[E / 2], uint32_t t, uint32_t gate_rows, int c, int left, float alpha,
                                        Red& red, int& turn, Read read) {
  using R = Row<VEC, E, FULL>;
  const int D = static_cast<int>(f.width);
  bool go = true;
  if (f.o != nullptr) {
    const float2 post = held_stat<VEC, E, FULL>(f.post, D, f.eps, n, left, red, turn);
    if (RING && f.post != kNone && blockDim.x > 32) go = read();
    if (threadIdx.x == 0 && f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = post;
    held_affine<RING, VEC, E, FULL>(n, f.post, post, f.w_post, par.w_post, f.b_post, par.b_post, c, left);
    const Pair a = both(alpha);
    if (f.gate != nullptr) {
      Pair g[E / 2];
      if (RING && par.gate != 0)
        param<RING, VEC, E, FULL>(nullptr, par.gate, c, left, g);
      else
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
  if (RING && !(f.o != nullptr && f.post != kNone && blockDim.x > 32)) {
    if (f.pre == kNone || blockDim.x == 32) team_sync();
    go = read();
  }
  if (threadIdx.x == 0 && f.stat_pre != nullptr) reinterpret_cast<float2*>(f.stat_pre)[t] = pre;
  if (f.h == nullptr && f.hq == nullptr) return go;
  held_affine<RING, VEC, E, FULL>(x, f.pre, pre, f.w_pre, par.w_pre, f.b_pre, par.b_pre, c, left);
  if (f.h != nullptr) R::store(static_cast<TB*>(f.h) + t * f.ld_h + c, left, x);
  if (f.hq != nullptr) {
    if (f.h_fmt == 0)
      emit_row<0, VEC, E>(f, x, t, c, left);
    else
      emit_row<1, VEC, E>(f, x, t, c, left);
  }
  return go;
}

// A row per CTA (or per warp), loaded straight into registers.
template <typename TS, typename TB, int VEC, int E, bool FULL>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormFwd f, int row_ctas, uint32_t gate_rows) {
  using R = Row<VEC, E, FULL>;
  __shared__ Red red;
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
  one_row<TS, TB, VEC, E, FULL, false>(f, Shared{}, x, n, t, gate_rows, c, left, f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f, red, turn, [] { return true; });
}

// Many rows: one CTA per SM, of several teams that take rows in turn (team threadIdx.y of CTA p: rows of every
// (p, team) apart). Asynchronous bulk copies bring a team's next rows into its ring in shared memory while the present
// one is worked on, and the parameters are kept in shared memory once for all teams: read from L1 next to the rings,
// which leave it some 30 KB, half of them missed (16384 x 4096: 110 us, in either form of the loads; TODO).
template <typename TS, typename TB, int E, bool FULL, int MOST>
__global__ void __launch_bounds__(MOST, 1) norm_fwd_ring_kernel(const NormFwd f, uint32_t gate_rows, int stages) {
  using R = Row<4, E, FULL>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Red reds[kMostTeams];
  __shared__ __align__(8) uint64_t bars[kMostTeams][kMaxStages];
  __shared__ volatile int fail[kMostTeams][2];  // rows in turn, so that no wait of the next row is taken for this one's
  const int team = threadIdx.y, teams = blockDim.y;
  const int D = static_cast<int>(f.width), c = R::first(threadIdx.x >> 5, threadIdx.x & 31), left = D - c;
  const uint32_t r_bytes = D * sizeof(TS), o_bytes = f.o != nullptr ? D * sizeof(TB) : 0u, bytes = r_bytes + o_bytes;
  const uint32_t bar0 = smem_u32(bars[team]), ring0 = team * stages * bytes;
  Red& red = reds[team];
  volatile int* failed = fail[team];
  if (blockDim.x > 32) red.clear();
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, 1);
    failed[0] = failed[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto fetch = [&](uint32_t t, int s) {  // (a team's thread 0)
    const uint32_t dst = smem_u32(smem) + ring0 + s * bytes;
    mbar_arrive_expect_tx(bar0 + 8 * s, bytes);
    bulk_load(dst, static_cast<const TS*>(f.r) + t * f.ld_r, r_bytes, bar0 + 8 * s);
    if (o_bytes != 0) bulk_load(dst + r_bytes, static_cast<const TB*>(f.o) + t * f.ld_o, o_bytes, bar0 + 8 * s);
  };
  const uint32_t T = static_cast<uint32_t>(f.tokens), t0 = blockIdx.x + team * gridDim.x, step = gridDim.x * teams;
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && t0 + s * static_cast<uint64_t>(step) < T; ++s) fetch(t0 + s * step, s);
  const int tid = team * blockDim.x + threadIdx.x, threads = blockDim.x * teams;
  Shared par{};
  {
    uint32_t at = teams * stages * bytes;
    auto keep = [&](const auto* p) {
      if (p == nullptr) return 0u;
      float* to = reinterpret_cast<float*>(smem + at);
      for (int i = tid; i < D; i += threads) to[i] = load(p + i);
      const uint32_t was = smem_u32(smem) + at;
      at += 4 * D;
      return was;
    };
    par.w_post = keep(f.w_post);
    par.b_post = keep(f.b_post);
    par.w_pre = keep(f.w_pre);
    par.b_pre = keep(f.b_pre);
    par.gate = gate_rows >= T ? keep(static_cast<const TB*>(f.gate)) : 0u;
  }
  if (f.hq != nullptr) fill_scales(f, blockIdx.x * static_cast<int64_t>(threads) + tid, static_cast<int64_t>(gridDim.x) * threads);
  __syncthreads();
  const float alpha = f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f;
  int turn = 0, stage = 0, odd = 0;
  uint32_t phase = 0;
  bool go = true;
  for (uint64_t row = t0; go && row < T; row += step) {
    const uint32_t t = static_cast<uint32_t>(row);
    // a wait that ran out is looked at behind this row's barrier, so that the team stops together
    if (!mbar_wait(bar0 + 8 * stage, phase, f.w, DEV_ERR_WAIT_PRODUCER)) failed[odd] = 1;
    const uint8_t* held = smem + ring0 + stage * bytes;
    Pair x[E / 2], n[E / 2];
    row_of<true, 4, E, FULL, TS>(held, 0, nullptr, 0, t, c, left, x);
    if (f.o != nullptr) row_of<true, 4, E, FULL, TB>(held, r_bytes, nullptr, 0, t, c, left, n);
    go = one_row<TS, TB, 4, E, FULL, true>(f, par, x, n, t, gate_rows, c, left, alpha, red, turn, [&] {
      if (failed[odd] != 0) return false;
      const uint64_t next = row + static_cast<uint64_t>(stages) * step;
      if (threadIdx.x == 0 && next < T) fetch(static_cast<uint32_t>(next), stage);
      return true;
    });
    odd ^= 1;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (!go && threadIdx.x == 0) {  // copies in flight land (microseconds) before the CTA can exit
    const unsigned long long w0 = globaltimer_ns();
    while (globaltimer_ns() - w0 < 200000ull) {
    }
  }
}

uint32_t gate_rows_of(const NormFwd& f) { return static_cast<uint32_t>(f.gate == nullptr || f.gate_rows > f.tokens ? f.tokens : f.gate_rows); }

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

// The ring kernel's shape: teams of a row each, and the rows each holds ahead; stages 0 where nothing fits.
struct RingPlan {
  int threads, teams, stages, bytes;
};

RingPlan ring_plan(const NormFwd& f, int64_t ss, int64_t bs, int columns) {
  RingPlan p{};
  p.threads = static_cast<int>((f.width + 32 * columns - 1) / (32 * columns)) * 32;
  p.teams = p.threads > 256 ? 1 : 768 / p.threads;  // (by registers: 80 a thread of 768, 128 of 512)
  if (p.teams > kMostTeams) p.teams = kMostTeams;
  int64_t params = 0;
  for (const float* q : {f.w_post, f.b_post, f.w_pre, f.b_pre}) params += q != nullptr ? 4 * f.width : 0;
  if (f.gate != nullptr && f.gate_rows >= f.tokens) params += 4 * f.width;
  const int64_t row = f.width * (ss + (f.o != nullptr ? bs : 0)), room = (kRingBytes - params) / (row * p.teams);
  p.stages = static_cast<int>(room < 0 ? 0 : room < kMaxStages ? room : kMaxStages);
  p.bytes = static_cast<int>(params + p.stages * p.teams * row);
  return p;
}

template <typename TS, typename TB, int E, bool FULL, int MOST>
cudaError_t launch_ring(const NormFwd& f, const RingPlan& p, cudaStream_t stream) {
  static bool done[64] = {};  // the limit is per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
    e = cudaFuncSetAttribute(norm_fwd_ring_kernel<TS, TB, E, FULL, MOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  NormFwd g = f;
  g.w = wait_ctl();
  if (g.w.err == nullptr) return cudaErrorInvalidDevice;
  return launch_pdl(norm_fwd_ring_kernel<TS, TB, E, FULL, MOST>, dim3(num_sms()), dim3(p.threads, p.teams), p.bytes, stream, g, gate_rows_of(f), p.stages);
}

template <typename TS, typename TB>
cudaError_t fwd_as(const NormFwd& f, cudaStream_t stream) {
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  const bool vec = f.width % 4 == 0 && rows_aligned(f.r, f.ld_r, ss, 4 * ss) && rows_aligned(f.r_out, f.ld_r_out, ss, 4 * ss) &&
                   rows_aligned(f.o, f.ld_o, bs, 4 * bs) && rows_aligned(f.h, f.ld_h, bs, 4 * bs) && rows_aligned(f.gate, f.ld_gate, bs, 4 * bs) &&
                   rows_aligned(f.w_post, 0, 4, 16) && rows_aligned(f.b_post, 0, 4, 16) && rows_aligned(f.w_pre, 0, 4, 16) && rows_aligned(f.b_pre, 0, 4, 16);
  // 16 elements per lane keep enough loads in flight for the memory's rate; with no more rows than a few per SM the
  // latency counts instead, and a row is spread over twice the lanes
  const bool few = f.tokens <= 2ll * num_sms();
  if (f.width <= 256 || (few && f.width <= 4096)) {
    if (!vec) return launch_rows<TS, TB, 1, 8, false>(f, stream);
    return f.width % 256 == 0 ? launch_rows<TS, TB, 4, 8, true>(f, stream) : launch_rows<TS, TB, 4, 8, false>(f, stream);
  }
  const bool vec16 = vec && f.width * ss % 16 == 0 && f.width * bs % 16 == 0 && rows_aligned(f.r, f.ld_r, ss, 16) && rows_aligned(f.o, f.ld_o, bs, 16);
  if (vec16 && !few && f.width >= 1024 && f.width <= 8192) {
    const RingPlan p = ring_plan(f, ss, bs, 16);
    if (p.stages > 0) {
      const bool full = f.width % 512 == 0;
      if (p.threads <= 256) return full ? launch_ring<TS, TB, 16, true, 768>(f, p, stream) : launch_ring<TS, TB, 16, false, 768>(f, p, stream);
      return full ? launch_ring<TS, TB, 16, true, 512>(f, p, stream) : launch_ring<TS, TB, 16, false, 512>(f, p, stream);
    }
  }
  if (f.width <= 8192) {
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
