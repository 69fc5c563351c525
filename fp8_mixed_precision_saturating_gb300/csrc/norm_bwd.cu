// norm_bwd.cu -- backward of the norms around a block with its gate and the residual's scale (HBM-bound).
//
// With g the gradient at r' and D the width:
//   norm'(dy; x):  dz = dy w,  dx = rstd (dz - z mean(dz z) - [layer] mean(dz)),
//                  dw = sum_t dy z,  db = sum_t dy
//   g = dr_out + norm_pre'(dh; r');  dr = alpha g;  dalpha = sum g r
//   dn = gate g;  dgate = sum over the gate's rows of g n;  do = norm_post'(dn; o)
#include "norm.cuh"

namespace fp8gb {
namespace {

using namespace norms;

// CTA p takes the consecutive tokens [p R, (p + 1) R) and leaves its share of every column sum in
// its own rows of the workspace: 4 rows for the parameters, then 2 for the gate gradient of the
// groups that it shares with its neighbours (its first group, its last). A group inside one CTA's
// tokens is written out by that CTA alone. A second kernel adds the shares up in CTA order.
constexpr int kPart = 6;

// Any width and alignment: the row read again for every pass over it, the column sums in the
// workspace (which its CTA alone touches).
template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) norm_bwd_any_kernel(const NormFwd f, const NormBwd b, float* part, double* part_alpha,
                                                           int64_t rows_per) {
  __shared__ float2 red[2][32];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const float alpha = f.res_scale != nullptr ? *f.res_scale : 1.0f;
  const int64_t D = f.width, t0 = blockIdx.x * rows_per, t1 = min(t0 + rows_per, f.tokens);
  const float inv = 1.0f / static_cast<float>(D);
  float* mine = part + static_cast<int64_t>(blockIdx.x) * kPart * D;
  for (int64_t c = threadIdx.x; c < kPart * D; c += kThreads) mine[c] = 0.0f;
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
      for (int64_t c = threadIdx.x; c < D; c += kThreads) {
        const float dz = f.w_pre != nullptr ? load(dh + c) * f.w_pre[c] : load(dh + c);
        a += dz;
        q = fmaf(dz, zpre(c), q);
      }
      s1 = cta_sum2(make_float2(a, q), red, turn, kThreads / 32);
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
      for (int64_t c = threadIdx.x; c < D; c += kThreads) {
        float dz = grad(c);
        if (gate != nullptr) dz *= load(gate + c);
        if (f.w_post != nullptr) dz *= f.w_post[c];
        a += dz;
        q = fmaf(dz, (load(o + c) - post.x) * post.y, q);
      }
      s2 = cta_sum2(make_float2(a, q), red, turn, kThreads / 32);
    }
    const bool whole = f.gate != nullptr && grp * f.gate_rows >= t0 && (min((grp + 1) * f.gate_rows, f.tokens) <= t1);
    const bool last = f.gate != nullptr && (t + 1 == t1 || (t + 1) / f.gate_rows != grp);
    const int slot = f.gate != nullptr && grp != t0 / f.gate_rows ? 5 : 4;
    for (int64_t c = threadIdx.x; c < D; c += kThreads) {
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
    __shared__ double sums[kThreads];
    sums[threadIdx.x] = dalpha;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int i = 0; i < kThreads; ++i) s += sums[i];
      part_alpha[blockIdx.x] = s;
    }
  }
}

// ---------------------------------------------------------------------------------------
// A row in the registers of a CTA, the next rows on their way to shared memory
// ---------------------------------------------------------------------------------------
// Every input is read once, from a ring of rows that asynchronous bulk copies fill ahead (RING: rows of whole
// 16 bytes) or from global memory. A thread holds the same I items of VEC columns of every row, so the column
// sums stay in its registers over all of the CTA's tokens.
//   pass 1: dz and z of the norm before the next block; its two row sums; dw_pre, db_pre
//   pass 2: g, so dr and dalpha; dn, dgate, dw_post, db_post; dz and z of the norm after the block; its row sums
//   pass 3: do
constexpr int kMaxStages = 4;

struct Ring {
  int stages, bytes;            // rows held, bytes of one
  int dh, r_out, dr_out, o, r;  // each tensor's place in a row; -1: not there
};

template <int VEC>
__device__ __forceinline__ void store_part(float* p, const float (&v)[VEC]) {  // (D % 4 == 0 where VEC == 4)
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *p = v[0];
}

// VEC elements of a row at column c: from the ring's copy, or from global memory.
template <bool RING, int VEC, typename T>
__device__ __forceinline__ void item(const uint8_t* held, int at, const void* base, int64_t ld, int64_t t, int c, float (&v)[VEC]) {
  if constexpr (RING) {
    const T* p = reinterpret_cast<const T*>(held + at) + c;
    if constexpr (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
      unpack4(*reinterpret_cast<const uint2*>(p), v);
    }
  } else {
    load_stream<VEC>(static_cast<const T*>(base) + t * ld + c, v);
  }
}

// WHAT: 0 weights' sums only, 1 the gate's too, 2 the gate's and the biases', 3 the biases'.
template <typename TS, typename TB, int VEC, int I, bool RING, int WHAT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormFwd f, const NormBwd b, float* part, double* part_alpha, int64_t rows_per, const Ring ring) {
  constexpr bool GATE = WHAT == 1 || WHAT == 2, BIAS = WHAT >= 2;
  extern __shared__ __align__(16) uint8_t rows_smem[];
  __shared__ float2 red[2][32];
  __shared__ double red_alpha[16];
  __shared__ __align__(8) uint64_t bars[kMaxStages];
  const int D = static_cast<int>(f.width), step = blockDim.x * VEC, c0 = threadIdx.x * VEC, warps = blockDim.x >> 5;
  const int64_t t0 = blockIdx.x * rows_per, t1 = min(t0 + rows_per, f.tokens);
  const uint32_t bar0 = smem_u32(bars);
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < ring.stages; ++s) mbar_init(bar0 + 8 * s, 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();

  auto fetch = [&](int64_t t) {  // (thread 0) row t's inputs into its stage
    const int s = static_cast<int>((t - t0) % ring.stages);
    const uint32_t dst = smem_u32(rows_smem) + s * ring.bytes, bar = bar0 + 8 * s;
    const uint32_t nb = D * sizeof(TB), ns = D * sizeof(TS);
    mbar_arrive_expect_tx(bar, ring.bytes);
    if (ring.dh >= 0) bulk_load(dst + ring.dh, static_cast<const TB*>(b.dh) + t * b.ld_dh, nb, bar);
    if (ring.r_out >= 0) bulk_load(dst + ring.r_out, static_cast<const TS*>(f.r_out) + t * f.ld_r_out, ns, bar);
    if (ring.dr_out >= 0) bulk_load(dst + ring.dr_out, static_cast<const TS*>(b.dr_out) + t * b.ld_dr_out, ns, bar);
    if (ring.o >= 0) bulk_load(dst + ring.o, static_cast<const TB*>(f.o) + t * f.ld_o, nb, bar);
    if (ring.r >= 0) bulk_load(dst + ring.r, static_cast<const TS*>(f.r) + t * f.ld_r, ns, bar);
  };
  if (RING && threadIdx.x == 0)
    for (int s = 0; s < ring.stages && t0 + s < t1; ++s) fetch(t0 + s);

  int turn = 0;
  const float alpha = f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f, inv = 1.0f / static_cast<float>(D);
  float aw_pre[I][VEC], aw_post[I][VEC], ag[GATE ? I : 1][VEC], ab_pre[BIAS ? I : 1][VEC], ab_post[BIAS ? I : 1][VEC];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      aw_pre[i][j] = aw_post[i][j] = 0.0f;
      if constexpr (GATE) ag[i][j] = 0.0f;
      if constexpr (BIAS) ab_pre[i][j] = ab_post[i][j] = 0.0f;
    }
  // sum g r cancels (its terms have both signs), so the rounding of its running sum is kept: hi + lo
  float al_hi = 0.0f, al_lo = 0.0f;
  const bool back = b.dh != nullptr, normed = back && f.pre != kNone, block = f.o != nullptr;
  float* mine = part + static_cast<int64_t>(blockIdx.x) * kPart * D;
  bool ok = true;
  for (int64_t t = t0; t < t1; ++t) {
    const uint8_t* held = nullptr;
    if constexpr (RING) {
      const int s = static_cast<int>((t - t0) % ring.stages);
      ok = mbar_wait(bar0 + 8 * s, static_cast<uint32_t>((t - t0) / ring.stages) & 1u, f.w, DEV_ERR_WAIT_PRODUCER);
      ok = __syncthreads_or(!ok) == 0;
      if (!ok) break;  // a wait ran out: the CTA stops together
      held = rows_smem + s * ring.bytes;
    }
    const float2 pre = normed ? __ldg(reinterpret_cast<const float2*>(f.stat_pre) + t) : make_float2(0.0f, 1.0f);
    const float2 post = f.post != kNone ? __ldg(reinterpret_cast<const float2*>(f.stat_post) + t) : make_float2(0.0f, 1.0f);
    const int64_t grp = f.gate != nullptr ? t / f.gate_rows : 0;
    const TB* gate = f.gate != nullptr ? static_cast<const TB*>(f.gate) + grp * f.ld_gate : nullptr;
    float dz[I][VEC], z[I][VEC];
    float2 s1 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = c0 + i * step;
#pragma unroll
      for (int j = 0; j < VEC; ++j) dz[i][j] = z[i][j] = 0.0f;
      if (c < D && back) {
        float dy[VEC], w[VEC];
        item<RING, VEC, TB>(held, ring.dh, b.dh, b.ld_dh, t, c, dy);
        if (normed) item<RING, VEC, TS>(held, ring.r_out, f.r_out, f.ld_r_out, t, c, z[i]);
        if (f.w_pre != nullptr) load_param<VEC>(f.w_pre + c, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          z[i][j] = normed ? (z[i][j] - pre.x) * pre.y : 0.0f;
          aw_pre[i][j] = fmaf(dy[j], z[i][j], aw_pre[i][j]);
          if constexpr (BIAS) ab_pre[i][j] += dy[j];
          dz[i][j] = f.w_pre != nullptr ? dy[j] * w[j] : dy[j];
          s1.x += dz[i][j];
          s1.y = fmaf(dz[i][j], z[i][j], s1.y);
        }
      }
    }
    if (normed) s1 = cta_sum2(s1, red, turn, warps);
    const float m1 = f.pre == kLayer && normed ? s1.x * inv : 0.0f, q1 = normed ? s1.y * inv : 0.0f;
    float2 s2 = make_float2(0.0f, 0.0f);
    float row_alpha = 0.0f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = c0 + i * step;
      if (c < D) {
        float g[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[j] = 0.0f;
        if (b.dr_out != nullptr) item<RING, VEC, TS>(held, ring.dr_out, b.dr_out, b.ld_dr_out, t, c, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[j] = fmaf(dz[i][j] - z[i][j] * q1 - m1, pre.y, g[j]);
        if (b.dres_scale != nullptr) {
          float r[VEC];
          item<RING, VEC, TS>(held, ring.r, f.r, f.ld_r, t, c, r);
#pragma unroll
          for (int j = 0; j < VEC; ++j) row_alpha = fmaf(g[j], r[j], row_alpha);
        }
        if (b.dr != nullptr) {
          float v[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[j] = g[j] * alpha;
          store_stream<VEC>(static_cast<TS*>(b.dr) + t * b.ld_dr + c, v);
        }
        if (block) {
          float x[VEC], gv[VEC], w[VEC], bp[VEC];
          item<RING, VEC, TB>(held, ring.o, f.o, f.ld_o, t, c, x);
          if (gate != nullptr) load_param<VEC>(gate + c, gv);
          if (f.w_post != nullptr) load_param<VEC>(f.w_post + c, w);
          if (GATE && f.b_post != nullptr) load_param<VEC>(f.b_post + c, bp);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float zo = (x[j] - post.x) * post.y;
            if constexpr (GATE) {
              float n = f.w_post != nullptr ? zo * w[j] : zo;
              if (f.b_post != nullptr) n += bp[j];
              ag[i][j] = fmaf(g[j], n, ag[i][j]);
            }
            const float dn = gate != nullptr ? g[j] * gv[j] : g[j];
            aw_post[i][j] = fmaf(dn, zo, aw_post[i][j]);
            if constexpr (BIAS) ab_post[i][j] += dn;
            z[i][j] = zo;
            dz[i][j] = f.w_post != nullptr ? dn * w[j] : dn;
            s2.x += dz[i][j];
            s2.y = fmaf(dz[i][j], zo, s2.y);
          }
        }
      }
    }
    {  // two-sum
      const float sum = __fadd_rn(al_hi, row_alpha), part2 = __fsub_rn(sum, al_hi);
      al_lo += __fadd_rn(__fsub_rn(al_hi, __fsub_rn(sum, part2)), __fsub_rn(row_alpha, part2));
      al_hi = sum;
    }
    if (block && f.post != kNone && b.dO != nullptr && warps > 1)
      s2 = cta_sum2(s2, red, turn, warps);
    else {
      s2 = warp_sum2(s2);  // (a CTA of one warp, or not needed)
      if constexpr (RING) __syncthreads();
    }
    // a barrier of this row is behind every read of its stage: the next row may land there
    if (RING && threadIdx.x == 0 && t + ring.stages < t1) fetch(t + ring.stages);
    if (b.dO != nullptr) {
      const float m2 = f.post == kLayer ? s2.x * inv : 0.0f, q2 = f.post != kNone ? s2.y * inv : 0.0f;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int c = c0 + i * step;
        if (c < D) {
          float v[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[j] = (dz[i][j] - z[i][j] * q2 - m2) * post.y;
          store_stream<VEC>(static_cast<TB*>(b.dO) + t * b.ld_do + c, v);
        }
      }
    }
    if constexpr (GATE) {
      if (t + 1 == t1 || (t + 1) / f.gate_rows != grp) {
        const bool whole = grp * f.gate_rows >= t0 && min((grp + 1) * f.gate_rows, f.tokens) <= t1;
        float* to = whole ? b.dgate + grp * D : mine + (grp == t0 / f.gate_rows ? 4 : 5) * static_cast<int64_t>(D);
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int c = c0 + i * step;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            if (c < D) to[c + j] = ag[i][j];
            ag[i][j] = 0.0f;
          }
        }
      }
    }
  }
  if (RING && !ok && threadIdx.x == 0) {  // copies in flight land (microseconds) before the CTA can exit
    const unsigned long long w0 = globaltimer_ns();
    while (globaltimer_ns() - w0 < 200000ull) {
    }
  }
  auto leave = [&](int k, const float(&a)[I][VEC]) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = c0 + i * step;
      if (c < D) store_part<VEC>(mine + k * static_cast<int64_t>(D) + c, a[i]);
    }
  };
  if (b.dw_pre != nullptr) leave(0, aw_pre);
  if (b.dw_post != nullptr) leave(2, aw_post);
  if constexpr (BIAS) {
    leave(1, ab_pre);
    leave(3, ab_post);
  }
  if (b.dres_scale != nullptr) {
    double a = static_cast<double>(al_hi) + static_cast<double>(al_lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if ((threadIdx.x & 31) == 0) red_alpha[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < warps; ++w) a += red_alpha[w];
      part_alpha[blockIdx.x] = a;
    }
  }
}

// Column sums over CTAs' partial rows: 32 columns per CTA; its 8 warps take consecutive ranges of the
// partial rows, and their sums are added in warp order. blockIdx.y 0 .. 3: the parameters (and alpha);
// 3 + p for p >= 1: the gate group that CTAs p - 1 and p share, if CTA p - 1 holds its first token.
__global__ void __launch_bounds__(kThreads) norm_bwd_reduce_kernel(const NormFwd f, const NormBwd b, const float* part,
                                                                   const double* part_alpha, int64_t rows_per, int ctas) {
  __shared__ float sums[8][32];
  pdl_wait();
  pdl_trigger();
  const int64_t D = f.width, c = blockIdx.x * 32ll + (threadIdx.x & 31);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto add = [&](int q0, int q1, auto place, float* out) {  // out[c] = sum over q of the partial row place(q)
    float s = 0.0f;
    const int n = q1 - q0, e = q0 + n * (warp + 1) / 8;
    if (c < D) {
      int q = q0 + n * warp / 8;
      for (; q + 8 <= e; q += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = __ldcs(part + place(q + u) * D + c);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
      }
      for (; q < e; ++q) s += __ldcs(part + place(q) * D + c);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
#pragma unroll
      for (int w = 1; w < 8; ++w) s += sums[w][lane];
      out[c] = s;
    }
    __syncthreads();
  };
  if (blockIdx.y < 4) {
    const int k = blockIdx.y;
    float* out = k == 0 ? b.dw_pre : k == 1 ? b.db_pre : k == 2 ? b.dw_post : b.db_post;
    if (out != nullptr) add(0, ctas, [=](int q) { return static_cast<int64_t>(q) * kPart + k; }, out);
    if (k == 0 && b.dres_scale != nullptr && blockIdx.x == 0 && warp == 0) {
      double s = 0.0;
      for (int p = lane; p < ctas; p += 32) s += part_alpha[p];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (lane == 0) *b.dres_scale = static_cast<float>(s);
    }
    return;
  }
  const int p = static_cast<int>(blockIdx.y) - 3;
  const int64_t first = p * rows_per;  // CTA p's first token
  const int64_t grp = first / f.gate_rows, ga = grp * f.gate_rows, ge = min(ga + f.gate_rows, f.tokens);
  if (ga == first || ga / rows_per != p - 1) return;
  const int last = static_cast<int>((ge - 1) / rows_per);
  add(p - 1, last + 1, [=](int q) { return static_cast<int64_t>(q) * kPart + (q * rows_per / f.gate_rows == grp ? 4 : 5); }, b.dgate + grp * D);
}

// The split of the tokens, from the sizes alone: CTAs of a row each, enough per SM for some 512 threads.
struct BwdPlan {
  int ctas, threads, per_sm;
  int64_t rows_per;
};

int items_of(int64_t width) { return width <= 2048 ? 2 : 4; }  // of 4 columns per thread

BwdPlan bwd_plan(int64_t tokens, int64_t width) {
  BwdPlan p;
  const int64_t per = 32 * 4 * items_of(width);
  p.threads = width <= 8192 ? static_cast<int>((width + per - 1) / per) * 32 : kThreads;
  p.per_sm = p.threads >= 512 ? 1 : p.threads >= 256 ? 2 : 4;
  const int64_t most = static_cast<int64_t>(p.per_sm) * num_sms();
  p.rows_per = (tokens + most - 1) / most;
  p.ctas = static_cast<int>((tokens + p.rows_per - 1) / p.rows_per);
  return p;
}

constexpr int kRingBytes = 216 * 1024;  // of an SM's shared memory

template <typename TS, typename TB, int VEC, int I, bool RING, int WHAT>
cudaError_t launch_kernel(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, const Ring& ring, cudaStream_t stream) {
  if constexpr (RING) {
    static bool done[64] = {};  // the limit is per device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
      e = cudaFuncSetAttribute(norm_bwd_kernel<TS, TB, VEC, I, RING, WHAT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
      if (e == cudaSuccess && dev < 64) done[dev] = true;
    }
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_bwd_kernel<TS, TB, VEC, I, RING, WHAT>, dim3(pl.ctas), dim3(pl.threads), RING ? ring.stages * ring.bytes : 0, stream, f, b, part,
                    part_alpha, pl.rows_per, ring);
}

template <typename TS, typename TB, int VEC, int I, bool RING>
cudaError_t launch_what(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, const Ring& ring, cudaStream_t stream) {
  const bool bias = b.db_pre != nullptr || b.db_post != nullptr;
  if (b.dgate != nullptr)
    return bias ? launch_kernel<TS, TB, VEC, I, RING, 2>(f, b, pl, part, part_alpha, ring, stream)
                : launch_kernel<TS, TB, VEC, I, RING, 1>(f, b, pl, part, part_alpha, ring, stream);
  return bias ? launch_kernel<TS, TB, VEC, I, RING, 3>(f, b, pl, part, part_alpha, ring, stream)
              : launch_kernel<TS, TB, VEC, I, RING, 0>(f, b, pl, part, part_alpha, ring, stream);
}

template <typename TS, typename TB>
cudaError_t bwd_as(const NormFwd& f, const NormBwd& b, void* ws, cudaStream_t stream) {
  const BwdPlan pl = bwd_plan(f.tokens, f.width);
  double* part_alpha = static_cast<double*>(ws);
  float* part = reinterpret_cast<float*>(part_alpha + pl.ctas + (pl.ctas & 1));
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  cudaError_t e;
  if (f.width > 8192) {
    e = launch_pdl(norm_bwd_any_kernel<TS, TB>, dim3(pl.ctas), dim3(kThreads), 0, stream, f, b, part, part_alpha, pl.rows_per);
  } else {
    Ring ring{0, 0, -1, -1, -1, -1, -1};
    bool vec = f.width * bs % 16 == 0 && f.width * ss % 16 == 0;
    auto place = [&](bool there, const void* p, int64_t ld, int64_t size, int& at) {
      if (!there) return;
      at = ring.bytes;
      ring.bytes += static_cast<int>(f.width * size);
      vec = vec && rows_aligned(p, ld, size, 16);
    };
    place(b.dh != nullptr, b.dh, b.ld_dh, bs, ring.dh);
    place(b.dh != nullptr && f.pre != kNone, f.r_out, f.ld_r_out, ss, ring.r_out);
    place(b.dr_out != nullptr, b.dr_out, b.ld_dr_out, ss, ring.dr_out);
    place(f.o != nullptr, f.o, f.ld_o, bs, ring.o);
    place(b.dres_scale != nullptr, f.r, f.ld_r, ss, ring.r);
    vec = vec && rows_aligned(f.gate, f.ld_gate, bs, 4 * bs) && rows_aligned(b.dr, b.ld_dr, ss, 4 * ss) && rows_aligned(b.dO, b.ld_do, bs, 4 * bs) &&
          rows_aligned(f.w_post, 0, 4, 16) && rows_aligned(f.b_post, 0, 4, 16) && rows_aligned(f.w_pre, 0, 4, 16);
    const bool two = items_of(f.width) == 2;
    if (vec) {
      const int64_t room = kRingBytes / pl.per_sm / ring.bytes;
      ring.stages = static_cast<int>(room < 1 ? 1 : room < kMaxStages ? room : kMaxStages);
      e = two ? launch_what<TS, TB, 4, 2, true>(f, b, pl, part, part_alpha, ring, stream)
              : launch_what<TS, TB, 4, 4, true>(f, b, pl, part, part_alpha, ring, stream);
    } else {
      e = two ? launch_what<TS, TB, 1, 8, false>(f, b, pl, part, part_alpha, ring, stream)
              : launch_what<TS, TB, 1, 16, false>(f, b, pl, part, part_alpha, ring, stream);
    }
  }
  if (e != cudaSuccess) return e;
  const bool split = b.dgate != nullptr && pl.ctas > 1;
  const dim3 grid(static_cast<unsigned>((f.width + 31) / 32), 4u + (split ? static_cast<unsigned>(pl.ctas - 1) : 0u));
  return launch_pdl(norm_bwd_reduce_kernel, grid, dim3(kThreads), 0, stream, f, b, part, part_alpha, pl.rows_per, pl.ctas);
}

}  // namespace

int64_t norm_bwd_workspace_bytes(const NormFwd& f) {
  if (f.tokens == 0 || f.width == 0) return 0;
  const int64_t ctas = bwd_plan(f.tokens, f.width).ctas;
  return ctas * kPart * f.width * 4 + (ctas + 1) / 2 * 16;
}

cudaError_t launch_norm_bwd(const NormFwd& f, const NormBwd& b, void* ws, cudaStream_t stream) {
  NormFwd g = f;
  g.w = wait_ctl();
  if (g.w.err == nullptr) return cudaErrorInvalidDevice;
  if (f.stream_f32)
    return f.block_f32 ? bwd_as<float, float>(g, b, ws, stream) : bwd_as<float, bf16>(g, b, ws, stream);
  return f.block_f32 ? bwd_as<bf16, float>(g, b, ws, stream) : bwd_as<bf16, bf16>(g, b, ws, stream);
}

}  // namespace fp8gb
