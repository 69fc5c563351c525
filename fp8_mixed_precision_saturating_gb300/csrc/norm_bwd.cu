// norm_bwd.cu -- backward of the norms around a block with its gate and the residual's scale (HBM-bound).
//
// With g the gradient at r' and D the width:
//   norm'(dy; x):  dz = dy w,  dx = rstd (dz - z mean(dz z) - [layer] mean(dz)),
//                  dw = sum_t dy z,  db = sum_t dy
//   g = dr_out + norm_pre'(dh; r');  dr = alpha g;  dalpha = sum g r
//   dn = gate g;  dgate = sum over the gate's rows of g n;  do = norm_post'(dn; o)
#include "norm_bwd.cuh"

namespace fp8gb {
namespace {

using namespace norms;

// Any width and alignment: the row read again for every pass over it, the column sums in the
// workspace (which its CTA alone touches). Bound by those sums' way through global memory, row by row:
// 8192 x 12288 bf16 4.4 ms, where the rows' bytes take 0.18.
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
// A row in the registers of a CTA
// ---------------------------------------------------------------------------------------
// Every input is read once. A thread holds the same E columns of every row, so the column sums stay in its registers
// over all of the CTA's tokens.
//   pass 1: dz and z of the norm before the next block; its row sums; dw_pre, db_pre
//   pass 2: g, so dr and dalpha; dz and z of the norm after the block; its row sums
// dgate, dw_post and db_post are all made of sum g z and sum g over the rows that share a gate: with n = z w + b and
// dn = gate g,  dgate = w sum g z + b sum g,  dw_post = sum over the gates of gate sum g z,  db_post likewise. So the
// rows add to those two sums alone, and they are spent where the gate's row changes.
//   pass 3: do
// SUM: sum dh and sum g are wanted (a bias's gradient, or the gate's where there is a bias). Bound by the latency of a
// row's loads and sums, with 15 to 20 warps on an SM: 16384 x 52 bf16 17 us, 4099 x 1537 47.6.
template <typename TS, typename TB, int VEC, int E, bool SUM>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormFwd f, const NormBwd b, float* part, double* part_alpha, int64_t rows_per) {
  // EARLY: all of a row's loads at once, an input that is not there as a row of no columns, so that no branch parts
  // them (16384 x 52 bf16: 26.3 -> 17.1 us; 4099 x 1537 in 8 columns a lane, fp32 stream: 50.9 -> 45.5). With 16 columns a lane the registers
  // are short, and single 16-bit elements take one each (4099 x 1537 bf16: 54.3 -> 62.8).
  constexpr bool EARLY = E == 8 && (VEC == 4 || sizeof(TS) == 4);
  using R = Row<VEC, E, false>;
  constexpr int H = E / 2;
  __shared__ Red red;
  __shared__ double red_alpha[16];
  const int D = static_cast<int>(f.width), warps = blockDim.x >> 5, c = R::first(threadIdx.x >> 5, threadIdx.x & 31), left = D - c;
  const int64_t t0 = blockIdx.x * rows_per, t1 = min(t0 + rows_per, f.tokens);
  if (warps > 1) red.clear();
  pdl_wait();
  pdl_trigger();

  int turn = 0;
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
  for (int64_t t = t0; t < t1; ++t) {
    if (f.gate != nullptr && t == grp_end) {
      ++grp;
      grp_end += f.gate_rows;
    }
    const float2 pre = normed ? __ldg(reinterpret_cast<const float2*>(f.stat_pre) + t) : make_float2(0.0f, 1.0f);
    const float2 post = f.post != kNone ? __ldg(reinterpret_cast<const float2*>(f.stat_post) + t) : make_float2(0.0f, 1.0f);
    Pair dz[H], z[H];
    Pair x_dr[EARLY ? H : 1], x_r[EARLY ? H : 1], x_o[EARLY ? H : 1];
    if constexpr (EARLY) {
      R::template load<true>(static_cast<const TB*>(b.dh) + t * b.ld_dh + c, back ? left : 0, dz);
      R::template load<true>(static_cast<const TS*>(f.r_out) + t * f.ld_r_out + c, normed ? left : 0, z);
      R::template load<true>(static_cast<const TS*>(b.dr_out) + t * b.ld_dr_out + c, b.dr_out != nullptr ? left : 0, x_dr);
      R::template load<true>(static_cast<const TB*>(f.o) + t * f.ld_o + c, block ? left : 0, x_o);
      R::template load<true>(static_cast<const TS*>(f.r) + t * f.ld_r + c, b.dres_scale != nullptr ? left : 0, x_r);
    }
    float m1 = 0.0f, q1 = 0.0f;
    if (back) {
      if constexpr (!EARLY) R::template load<true>(static_cast<const TB*>(b.dh) + t * b.ld_dh + c, left, dz);
      if constexpr (SUM) {
#pragma unroll
        for (int i = 0; i < H; ++i) ab_pre[i] = add2(ab_pre[i], dz[i]);
      }
      if (normed) {
        if constexpr (!EARLY) R::template load<true>(static_cast<const TS*>(f.r_out) + t * f.ld_r_out + c, left, z);
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
    auto take = [&](const auto& early, const auto* row) {  // the row's columns into z
      if constexpr (EARLY) {
#pragma unroll
        for (int i = 0; i < H; ++i) z[i] = early[i];
      } else {
        R::template load<true>(row + c, left, z);
      }
    };
    // dz, times rstd: the norm's share of g, the gradient at r'
    {
      const Pair rstd = both(pre.y);
      if (b.dr_out != nullptr) {
        take(x_dr, static_cast<const TS*>(b.dr_out) + t * b.ld_dr_out);
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = fma2(dz[i], rstd, z[i]);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = mul2(dz[i], rstd);
      }
    }
    R::clear(dz, left);
    if (b.dres_scale != nullptr) {
      take(x_r, static_cast<const TS*>(f.r) + t * f.ld_r);
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
      take(x_o, static_cast<const TB*>(f.o) + t * f.ld_o);
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
        leave<VEC, E, false, false>((whole ? b.dgate + grp * D : mine + (grp == grp0 ? 4 : 5) * static_cast<int64_t>(D)) + c, left, v);
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
        leave<VEC, E, false, true>(p, left, a);
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
  if (b.dw_pre != nullptr) leave<VEC, E, false, true>(mine + c, left, aw_pre);
  if constexpr (SUM) leave<VEC, E, false, true>(mine + D + c, left, ab_pre);
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

// Column sums over the parts' rows: 8 V columns per CTA (V = 4 where rows are whole 16 bytes). Its 16 warps take
// consecutive ranges of the parts, the four quarters of a warp every fourth one, so that some 1200 parts are three rounds
// of loads for a lane; the sums are added in this order whatever runs first. Bound by the latency of those rounds: 6 us
// for 456 parts of 1536 columns with 9 gate groups, behind 28 us for the parts (a warp a range, its lanes over columns:
// 10). blockIdx.y 0 .. 3: the parameters (and alpha); from 4 on: the gate groups that several parts share.
constexpr int kReduceWarps = 16, kBatch = 8;

template <int V>
struct Cols {
  float v[V];
};

template <int V>
__global__ void __launch_bounds__(32 * kReduceWarps) norm_bwd_reduce_kernel(const NormFwd f, const NormBwd b, const float* part,
                                                                            const double* part_alpha, int64_t rows_per, int parts) {
  __shared__ Cols<V> sums[kReduceWarps][8];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t D = f.width, c = (blockIdx.x * 8ll + (lane & 7)) * V;
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
      for (int q = q0 + n * warp / kReduceWarps + (lane >> 3); q < e; q += 4 * kBatch) {
        Cols<V> x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) x[u] = fetch(place(min(q + 4 * u, e - 1)));  // (past the range: its last row, not added)
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int j = 0; j < V; ++j) s.v[j] += q + 4 * u < e ? x[u].v[j] : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s.v[j] += __shfl_xor_sync(0xFFFFFFFFu, s.v[j], 8);
      s.v[j] += __shfl_xor_sync(0xFFFFFFFFu, s.v[j], 16);
    }
    if (lane < 8) sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && lane < 8 && c < D) {
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
    if (out != nullptr) add(0, parts, [=](int q) { return static_cast<int64_t>(q) * kPart + k; }, out);
    if (k == 0 && b.dres_scale != nullptr && blockIdx.x == 0 && warp == 0) {
      double s = 0.0;
      for (int p = lane; p < parts; p += 32) s += part_alpha[p];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (lane == 0) *b.dres_scale = static_cast<float>(s);
    }
    return;
  }
  // by groups where they are fewer than the parts, else by the parts' borders
  const int64_t groups = gate_groups(f);
  const bool by_group = groups < parts;
  for (int64_t i = blockIdx.y - 4; i < (by_group ? groups : parts - 1); i += gridDim.y - 4) {
    const int64_t grp = by_group ? i : (i + 1) * rows_per / f.gate_rows, ga = grp * f.gate_rows, ge = min(ga + f.gate_rows, f.tokens);
    const int first = static_cast<int>(ga / rows_per), last = static_cast<int>((ge - 1) / rows_per);
    if (first == last || (!by_group && first != i)) continue;  // one part's alone, or another border's
    // the group is the last one of the part that holds its first token, unless it is that part's first too
    const int slot = first * rows_per / f.gate_rows == grp ? 4 : 5;
    add(first, last + 1, [=](int q) { return static_cast<int64_t>(q) * kPart + (q == first ? slot : 4); }, b.dgate + grp * D);
  }
}

template <typename TS, typename TB, int VEC, int E>
cudaError_t launch_rows(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, cudaStream_t stream) {
  if (sums_wanted(f, b))
    return launch_pdl(norm_bwd_kernel<TS, TB, VEC, E, true>, dim3(pl.parts), dim3(pl.threads), 0, stream, f, b, part, part_alpha, pl.rows_per);
  return launch_pdl(norm_bwd_kernel<TS, TB, VEC, E, false>, dim3(pl.parts), dim3(pl.threads), 0, stream, f, b, part, part_alpha, pl.rows_per);
}

template <typename TS, typename TB>
cudaError_t bwd_as(const NormFwd& f, const NormBwd& b, void* ws, cudaStream_t stream) {
  const BwdPlan pl = bwd_plan(f.tokens, f.width);
  double* part_alpha = static_cast<double*>(ws);
  float* part = reinterpret_cast<float*>(part_alpha + pl.parts + (pl.parts & 1));
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  bool taken = false;
  cudaError_t e = launch_norm_bwd_ring(f, b, pl, part, part_alpha, stream, &taken);
  if (e != cudaSuccess) return e;
  if (taken) {
  } else if (f.width > 8192) {
    e = launch_pdl(norm_bwd_any_kernel<TS, TB>, dim3(pl.parts), dim3(kThreads), 0, stream, f, b, part, part_alpha, pl.rows_per);
  } else {
    const bool vec = f.width % 4 == 0 && rows_aligned(f.r, f.tokens, f.ld_r, ss, 4 * ss) && rows_aligned(f.r_out, f.tokens, f.ld_r_out, ss, 4 * ss) &&
                     rows_aligned(f.o, f.tokens, f.ld_o, bs, 4 * bs) && rows_aligned(f.gate, gate_groups(f), f.ld_gate, bs, 4 * bs) && rows_aligned(b.dh, f.tokens, b.ld_dh, bs, 4 * bs) &&
                     rows_aligned(b.dr_out, f.tokens, b.ld_dr_out, ss, 4 * ss) && rows_aligned(b.dr, f.tokens, b.ld_dr, ss, 4 * ss) && rows_aligned(b.dO, f.tokens, b.ld_do, bs, 4 * bs) &&
                     rows_aligned(f.w_post, 1, 0, 4, 16) && rows_aligned(f.b_post, 1, 0, 4, 16) && rows_aligned(f.w_pre, 1, 0, 4, 16);
    if (columns_of(f.width) == 8)
      e = vec ? launch_rows<TS, TB, 4, 8>(f, b, pl, part, part_alpha, stream) : launch_rows<TS, TB, 1, 8>(f, b, pl, part, part_alpha, stream);
    else
      e = vec ? launch_rows<TS, TB, 4, 16>(f, b, pl, part, part_alpha, stream) : launch_rows<TS, TB, 1, 16>(f, b, pl, part, part_alpha, stream);
  }
  if (e != cudaSuccess) return e;
  int64_t shared = 0;  // gate groups that may be shared
  if (b.dgate != nullptr && pl.parts > 1) {
    const int64_t groups = gate_groups(f);
    shared = groups < pl.parts ? groups : pl.parts - 1;
  }
  const int cols = f.width % 4 == 0 ? 32 : 8;
  const dim3 grid(static_cast<unsigned>((f.width + cols - 1) / cols), static_cast<unsigned>(4 + (shared < 32 ? shared : 32)));
  return launch_pdl(cols == 32 ? norm_bwd_reduce_kernel<4> : norm_bwd_reduce_kernel<1>, grid, dim3(32 * kReduceWarps), 0, stream, f, b, part, part_alpha,
                    pl.rows_per, pl.parts);
}

}  // namespace

int64_t norm_bwd_workspace_bytes(const NormFwd& f) {
  if (f.tokens == 0 || f.width == 0) return 0;
  const int64_t parts = bwd_plan(f.tokens, f.width).parts;
  return parts * kPart * f.width * 4 + (parts + 1) / 2 * 16;
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
