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
  __shared__ Red red;
  int turn = 0;
  red.clear();
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
      s1 = cta_sum(make_float2(a, q), red, turn);
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
      s2 = cta_sum(make_float2(a, q), red, turn);
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
// 16 bytes) or from global memory. A thread holds the same E columns of every row, so the column sums stay in its
// registers over all of the CTA's tokens.
//   pass 1: dz and z of the norm before the next block; its row sums; dw_pre, db_pre
//   pass 2: g, so dr and dalpha; dz and z of the norm after the block; its row sums
// dgate, dw_post and db_post are all made of sum g z and sum g over the rows that share a gate: with n = z w + b and
// dn = gate g,  dgate = w sum g z + b sum g,  dw_post = sum over the gates of gate sum g z,  db_post likewise. So the
// rows add to those two sums alone, and they are spent where the gate's row changes.
//   pass 3: do
struct Ring {
  int stages, bytes;            // rows held, bytes of one
  int dh, r_out, dr_out, o, r;  // each tensor's place in a row; -1: not there
};

// Column sums to the workspace (WIDE; they stay in L2 for the kernel that adds them up) or to dgate (aligned to 4 bytes only).
template <int VEC, int E, bool FULL, bool WIDE>
__device__ __forceinline__ void leave(float* p, int left, const Pair (&x)[E / 2]) {
  if constexpr (VEC == 4 && !WIDE) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float2 a = split(x[2 * i]), b = split(x[2 * i + 1]);
      if (FULL || 128 * i < left) {
        p[128 * i] = a.x;
        p[128 * i + 1] = a.y;
        p[128 * i + 2] = b.x;
        p[128 * i + 3] = b.y;
      }
    }
  } else if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float2 a = split(x[2 * i]), b = split(x[2 * i + 1]);
      if (FULL || 128 * i < left) *reinterpret_cast<float4*>(p + 128 * i) = make_float4(a.x, a.y, b.x, b.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 a = split(x[i]);
      if (64 * i < left) p[64 * i] = a.x;
      if (64 * i + 32 < left) p[64 * i + 32] = a.y;
    }
  }
}

// SUM: sum dh and sum g are wanted (a bias's gradient, or the gate's where there is a bias).
template <typename TS, typename TB, int VEC, int E, bool FULL, bool RING, bool SUM>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormFwd f, const NormBwd b, float* part, double* part_alpha, int64_t rows_per, const Ring ring) {
  using R = Row<VEC, E, FULL>;
  constexpr int H = E / 2;
  extern __shared__ __align__(16) uint8_t rows_smem[];
  __shared__ Red red;
  __shared__ double red_alpha[16];
  __shared__ __align__(8) uint64_t bars[kMaxStages];
  __shared__ volatile int failed[2];  // rows in turn, so that no wait of the next row is taken for this one's
  const int D = static_cast<int>(f.width), warps = blockDim.x >> 5, c = R::first(threadIdx.x >> 5, threadIdx.x & 31), left = D - c;
  const int64_t t0 = blockIdx.x * rows_per, t1 = min(t0 + rows_per, f.tokens);
  const uint32_t bar0 = smem_u32(bars);
  if (warps > 1) red.clear();
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < ring.stages; ++s) mbar_init(bar0 + 8 * s, 1);
      failed[0] = failed[1] = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();

  auto fetch = [&](int64_t t, int s) {  // (thread 0) row t's inputs into stage s
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
    for (int s = 0; s < ring.stages && t0 + s < t1; ++s) fetch(t0 + s, s);

  int turn = 0, stage = 0;
  uint32_t phase = 0;
  const float alpha = f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f, inv = 1.0f / static_cast<float>(D);
  Pair aw_pre[H], agz[H], ab_pre[SUM ? H : 1], ag[SUM ? H : 1];
  const Pair zero = both(0.0f);
#pragma unroll
  for (int i = 0; i < H; ++i) {
    aw_pre[i] = agz[i] = zero;
    if constexpr (SUM) ab_pre[i] = ag[i] = zero;
  }
  bool spent = false;  // this CTA's rows of dw_post and db_post hold earlier gates' shares
  // sum g r cancels (its terms have both signs), so the rounding of its running sum is kept: hi + lo
  float al_hi = 0.0f, al_lo = 0.0f;
  const bool back = b.dh != nullptr, normed = back && f.pre != kNone, block = f.o != nullptr;
  float* mine = part + static_cast<int64_t>(blockIdx.x) * kPart * D;
  int64_t grp = 0, grp_end = f.tokens;  // the gate's row, and the first token past its group
  if (f.gate != nullptr) {
    grp = t0 / f.gate_rows;
    grp_end = (grp + 1) * f.gate_rows;
  }
  const int64_t grp0 = grp;
  bool stop = false;
  for (int64_t t = t0; t < t1; ++t) {
    const uint8_t* held = nullptr;
    if constexpr (RING) {
      // a wait that ran out is looked at behind this row's barrier, so that the CTA stops together
      if (!mbar_wait(bar0 + 8 * stage, phase, f.w, DEV_ERR_WAIT_PRODUCER)) failed[(t - t0) & 1] = 1;
      held = rows_smem + stage * ring.bytes;
    }
    if (f.gate != nullptr && t == grp_end) {
      ++grp;
      grp_end += f.gate_rows;
    }
    const float2 pre = normed ? __ldg(reinterpret_cast<const float2*>(f.stat_pre) + t) : make_float2(0.0f, 1.0f);
    const float2 post = f.post != kNone ? __ldg(reinterpret_cast<const float2*>(f.stat_post) + t) : make_float2(0.0f, 1.0f);
    Pair dz[H], z[H];
    float m1 = 0.0f, q1 = 0.0f;
    if (back) {
      row_of<RING, VEC, E, FULL, TB>(held, ring.dh, b.dh, b.ld_dh, t, c, left, dz);
      if constexpr (SUM) {
#pragma unroll
        for (int i = 0; i < H; ++i) ab_pre[i] = add2(ab_pre[i], dz[i]);
      }
      if (normed) {
        row_of<RING, VEC, E, FULL, TS>(held, ring.r_out, f.r_out, f.ld_r_out, t, c, left, z);
        const Pair m = both(-pre.x), rstd = both(pre.y);
        if (f.pre == kLayer) {
#pragma unroll
          for (int i = 0; i < H; ++i) z[i] = add2(z[i], m);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          z[i] = mul2(z[i], rstd);
          aw_pre[i] = fma2(dz[i], z[i], aw_pre[i]);
        }
        if (f.w_pre != nullptr) {
          Pair w[H];
          R::template load<false>(f.w_pre + c, left, w);
#pragma unroll
          for (int i = 0; i < H; ++i) dz[i] = mul2(dz[i], w[i]);
        }
        Pair sq = zero;
#pragma unroll
        for (int i = 0; i < H; ++i) sq = fma2(dz[i], z[i], sq);
        if (f.pre == kLayer) {
          Pair sm = zero;
#pragma unroll
          for (int i = 0; i < H; ++i) sm = add2(sm, dz[i]);
          const float2 s = cta_sum(make_float2(sum2(sm), sum2(sq)), red, turn);
          m1 = s.x * inv;
          q1 = s.y * inv;
        } else {
          q1 = cta_sum(sum2(sq), red, turn) * inv;
        }
        const Pair q = both(-q1);
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = fma2(z[i], q, dz[i]);
        if (f.pre == kLayer) {
          const Pair mm = both(-m1);
#pragma unroll
          for (int i = 0; i < H; ++i) dz[i] = add2(dz[i], mm);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < H; ++i) dz[i] = zero;
    }
    // dz, times rstd: the norm's share of g, the gradient at r'
    {
      const Pair rstd = both(pre.y);
      if (b.dr_out != nullptr) {
        row_of<RING, VEC, E, FULL, TS>(held, ring.dr_out, b.dr_out, b.ld_dr_out, t, c, left, z);
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = fma2(dz[i], rstd, z[i]);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = mul2(dz[i], rstd);
      }
    }
    R::clear(dz, left);
    if (b.dres_scale != nullptr) {
      row_of<RING, VEC, E, FULL, TS>(held, ring.r, f.r, f.ld_r, t, c, left, z);
      Pair s = zero;
#pragma unroll
      for (int i = 0; i < H; ++i) s = fma2(dz[i], z[i], s);
      const float a = sum2(s), sum = __fadd_rn(al_hi, a), took = __fsub_rn(sum, al_hi);  // two-sum
      al_lo += __fadd_rn(__fsub_rn(al_hi, __fsub_rn(sum, took)), __fsub_rn(a, took));
      al_hi = sum;
    }
    if (b.dr != nullptr) {
      const Pair a = both(alpha);
#pragma unroll
      for (int i = 0; i < H; ++i) z[i] = mul2(dz[i], a);
      R::store(static_cast<TS*>(b.dr) + t * b.ld_dr + c, left, z);
    }
    float m2 = 0.0f, q2 = 0.0f;
    if (block) {
      row_of<RING, VEC, E, FULL, TB>(held, ring.o, f.o, f.ld_o, t, c, left, z);
      if (f.post != kNone) {
        if (f.post == kLayer) {
          const Pair m = both(-post.x);
#pragma unroll
          for (int i = 0; i < H; ++i) z[i] = add2(z[i], m);
        }
        const Pair rstd = both(post.y);
#pragma unroll
        for (int i = 0; i < H; ++i) z[i] = mul2(z[i], rstd);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) agz[i] = fma2(dz[i], z[i], agz[i]);
      if constexpr (SUM) {
#pragma unroll
        for (int i = 0; i < H; ++i) ag[i] = add2(ag[i], dz[i]);
      }
      if (f.gate != nullptr) {
        Pair g[H];
        R::template load<false>(static_cast<const TB*>(f.gate) + grp * f.ld_gate + c, left, g);
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = mul2(dz[i], g[i]);
      }
      if (f.w_post != nullptr) {
        Pair w[H];
        R::template load<false>(f.w_post + c, left, w);
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = mul2(dz[i], w[i]);
      }
    }
    if (block && f.post != kNone && b.dO != nullptr) {
      Pair sq = zero;
#pragma unroll
      for (int i = 0; i < H; ++i) sq = fma2(dz[i], z[i], sq);
      if (f.post == kLayer) {
        Pair sm = zero;
#pragma unroll
        for (int i = 0; i < H; ++i) sm = add2(sm, dz[i]);
        const float2 s = cta_sum(make_float2(sum2(sm), sum2(sq)), red, turn);
        m2 = s.x * inv;
        q2 = s.y * inv;
      } else {
        q2 = cta_sum(sum2(sq), red, turn) * inv;
      }
      if (RING && warps == 1) __syncthreads();  // (its sum needs no barrier, its stage does)
    } else if constexpr (RING) {
      __syncthreads();
    }
    if constexpr (RING) {
      // a barrier of this row is behind every read of its stage: a later row may land there
      stop = failed[(t - t0) & 1] != 0;
      if (stop) break;
      if (threadIdx.x == 0 && t + ring.stages < t1) fetch(t + ring.stages, stage);
      if (++stage == ring.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (b.dO != nullptr) {
      if (f.post != kNone) {
        const Pair q = both(-q2), rstd = both(post.y);
        if (f.post == kLayer) {
          const Pair mm = both(-m2);
#pragma unroll
          for (int i = 0; i < H; ++i) dz[i] = add2(dz[i], mm);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = mul2(fma2(z[i], q, dz[i]), rstd);
      }
      R::store(static_cast<TB*>(b.dO) + t * b.ld_do + c, left, dz);
    }
    if (block && (t + 1 == t1 || (f.gate != nullptr && t + 1 == grp_end))) {
      if (b.dgate != nullptr) {
        const bool whole = grp_end - f.gate_rows >= t0 && min(grp_end, f.tokens) <= t1;
        Pair v[H];
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = agz[i];
        if (f.w_post != nullptr) {
          R::template load<false>(f.w_post + c, left, v);
#pragma unroll
          for (int i = 0; i < H; ++i) v[i] = mul2(v[i], agz[i]);
        }
        if constexpr (SUM) {
          if (f.b_post != nullptr) {
            Pair p[H];
            R::template load<false>(f.b_post + c, left, p);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = fma2(p[i], ag[i], v[i]);
          }
        }
        leave<VEC, E, FULL, false>((whole ? b.dgate + grp * D : mine + (grp == grp0 ? 4 : 5) * static_cast<int64_t>(D)) + c, left, v);
      }
      auto spend = [&](int k, Pair(&a)[H]) {  // gate times the sum, onto what earlier gates left
        Pair v[H];
        float* p = mine + k * static_cast<int64_t>(D) + c;
        if (f.gate != nullptr) {
          R::template load<false>(static_cast<const TB*>(f.gate) + grp * f.ld_gate + c, left, v);
#pragma unroll
          for (int i = 0; i < H; ++i) a[i] = mul2(a[i], v[i]);
        }
        if (spent) {
          R::template load<true>(p, left, v);
#pragma unroll
          for (int i = 0; i < H; ++i) a[i] = add2(a[i], v[i]);
        }
        leave<VEC, E, FULL, true>(p, left, a);
#pragma unroll
        for (int i = 0; i < H; ++i) a[i] = zero;
      };
      if (b.dw_post != nullptr) spend(2, agz);
      if constexpr (SUM) {
        if (b.db_post != nullptr) spend(3, ag);
      }
      spent = true;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        agz[i] = zero;
        if constexpr (SUM) ag[i] = zero;
      }
    }
  }
  if (RING && threadIdx.x == 0 && stop) {  // copies in flight land (microseconds) before the CTA can exit
    const unsigned long long w0 = globaltimer_ns();
    while (globaltimer_ns() - w0 < 200000ull) {
    }
  }
  if (b.dw_pre != nullptr) leave<VEC, E, FULL, true>(mine + c, left, aw_pre);
  if constexpr (SUM) leave<VEC, E, FULL, true>(mine + D + c, left, ab_pre);
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

// Column sums over CTAs' partial rows: 32 V columns per CTA (V = 4 where rows are whole 16 bytes); its 16 warps take
// consecutive ranges of the partial rows, and their sums are added in warp order. blockIdx.y 0 .. 3: the parameters
// (and alpha); from 4 on: the gate groups that several CTAs share.
constexpr int kReduceWarps = 16;

template <int V>
struct Cols {
  float v[V];
};

template <int V>
__global__ void __launch_bounds__(32 * kReduceWarps) norm_bwd_reduce_kernel(const NormFwd f, const NormBwd b, const float* part,
                                                                            const double* part_alpha, int64_t rows_per, int ctas) {
  __shared__ Cols<V> sums[kReduceWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t D = f.width, c = (blockIdx.x * 32ll + lane) * V;
  auto fetch = [&](int64_t row) {
    Cols<V> x;
    if constexpr (V == 4) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(part + row * D + c));
      x.v[0] = t.x, x.v[1] = t.y, x.v[2] = t.z, x.v[3] = t.w;
    } else {
      x.v[0] = __ldcg(part + row * D + c);
    }
    return x;
  };
  auto add = [&](int q0, int q1, auto place, float* out) {  // out[c] = sum over q of the partial row place(q)
    Cols<V> s = {};
    const int n = q1 - q0, e = q0 + n * (warp + 1) / kReduceWarps;
    if (c < D) {
      int q = q0 + n * warp / kReduceWarps;
      for (; q + 8 <= e; q += 8) {
        Cols<V> x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = fetch(place(q + u));
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int j = 0; j < V; ++j) s.v[j] += x[u].v[j];
      }
      for (; q < e; ++q) {
        const Cols<V> x = fetch(place(q));
#pragma unroll
        for (int j = 0; j < V; ++j) s.v[j] += x.v[j];
      }
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
#pragma unroll
      for (int w = 1; w < kReduceWarps; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) s.v[j] += sums[w][lane].v[j];
#pragma unroll
      for (int j = 0; j < V; ++j) out[c + j] = s.v[j];
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
  // by groups where they are fewer than the CTAs, else by the CTAs' borders
  const int64_t groups = (f.tokens + f.gate_rows - 1) / f.gate_rows;
  const bool by_group = groups < ctas;
  for (int64_t i = blockIdx.y - 4; i < (by_group ? groups : ctas - 1); i += gridDim.y - 4) {
    const int64_t grp = by_group ? i : (i + 1) * rows_per / f.gate_rows, ga = grp * f.gate_rows, ge = min(ga + f.gate_rows, f.tokens);
    const int first = static_cast<int>(ga / rows_per), last = static_cast<int>((ge - 1) / rows_per);
    if (first == last || (!by_group && first != i)) continue;  // one CTA's alone, or another border's
    // the group is the last one of the CTA that holds its first token, unless it is that CTA's first too
    const int slot = first * rows_per / f.gate_rows == grp ? 4 : 5;
    add(first, last + 1, [=](int q) { return static_cast<int64_t>(q) * kPart + (q == first ? slot : 4); }, b.dgate + grp * D);
  }
}

// The split of the tokens, from the sizes alone: CTAs of a row each, enough per SM for some 512 threads.
struct BwdPlan {
  int ctas, threads, per_sm;
  int64_t rows_per;
};

int columns_of(int64_t width) { return width <= 2048 ? 8 : 16; }  // per thread

BwdPlan bwd_plan(int64_t tokens, int64_t width) {
  BwdPlan p;
  const int64_t per = 32 * columns_of(width);
  p.threads = width <= 8192 ? static_cast<int>((width + per - 1) / per) * 32 : kThreads;
  p.per_sm = p.threads > 292 ? 1 : p.threads > 195 ? 2 : p.threads > 146 ? 3 : 4;  // (some 112 registers each)
  const int64_t most = static_cast<int64_t>(p.per_sm) * num_sms();
  p.rows_per = (tokens + most - 1) / most;
  p.ctas = static_cast<int>((tokens + p.rows_per - 1) / p.rows_per);
  return p;
}

template <typename TS, typename TB, int VEC, int E, bool FULL, bool RING, bool SUM>
cudaError_t launch_kernel(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, const Ring& ring, cudaStream_t stream) {
  if constexpr (RING) {
    static bool done[64] = {};  // the limit is per device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
      e = cudaFuncSetAttribute(norm_bwd_kernel<TS, TB, VEC, E, FULL, RING, SUM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
      if (e == cudaSuccess && dev < 64) done[dev] = true;
    }
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_bwd_kernel<TS, TB, VEC, E, FULL, RING, SUM>, dim3(pl.ctas), dim3(pl.threads), RING ? ring.stages * ring.bytes : 0, stream, f, b, part,
                    part_alpha, pl.rows_per, ring);
}

template <typename TS, typename TB, int VEC, int E, bool FULL, bool RING>
cudaError_t launch_sums(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, const Ring& ring, cudaStream_t stream) {
  if (b.db_pre != nullptr || b.db_post != nullptr || (b.dgate != nullptr && f.b_post != nullptr))
    return launch_kernel<TS, TB, VEC, E, FULL, RING, true>(f, b, pl, part, part_alpha, ring, stream);
  return launch_kernel<TS, TB, VEC, E, FULL, RING, false>(f, b, pl, part, part_alpha, ring, stream);
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
    const bool eight = columns_of(f.width) == 8;
    if (vec) {
      const int64_t room = kRingBytes / pl.per_sm / ring.bytes;
      ring.stages = static_cast<int>(room < 1 ? 1 : room < kMaxStages ? room : kMaxStages);
      const bool full = f.width % (eight ? 256 : 512) == 0;
      e = eight ? (full ? launch_sums<TS, TB, 4, 8, true, true>(f, b, pl, part, part_alpha, ring, stream)
                        : launch_sums<TS, TB, 4, 8, false, true>(f, b, pl, part, part_alpha, ring, stream))
                : (full ? launch_sums<TS, TB, 4, 16, true, true>(f, b, pl, part, part_alpha, ring, stream)
                        : launch_sums<TS, TB, 4, 16, false, true>(f, b, pl, part, part_alpha, ring, stream));
    } else {
      e = eight ? launch_sums<TS, TB, 1, 8, false, false>(f, b, pl, part, part_alpha, ring, stream)
              : launch_sums<TS, TB, 1, 16, false, false>(f, b, pl, part, part_alpha, ring, stream);
    }
  }
  if (e != cudaSuccess) return e;
  int64_t shared = 0;  // gate groups that may be shared
  if (b.dgate != nullptr && pl.ctas > 1) {
    const int64_t groups = (f.tokens + f.gate_rows - 1) / f.gate_rows;
    shared = groups < pl.ctas ? groups : pl.ctas - 1;
  }
  const int cols = f.width % 4 == 0 ? 128 : 32;
  const dim3 grid(static_cast<unsigned>((f.width + cols - 1) / cols), static_cast<unsigned>(4 + (shared < 32 ? shared : 32)));
  return launch_pdl(cols == 128 ? norm_bwd_reduce_kernel<4> : norm_bwd_reduce_kernel<1>, grid, dim3(32 * kReduceWarps), 0, stream, f, b, part, part_alpha,
                    pl.rows_per, pl.ctas);
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
