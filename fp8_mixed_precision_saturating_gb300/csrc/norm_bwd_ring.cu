// norm_bwd_ring.cu -- backward of the norms around a block for the whole of a training step's gradients (HBM-bound: 6
// passes over the rows, 7 with the residual scale's gradient: 12 to 14 bytes per element in bf16). The formulas and the
// sums' way: norm_bwd.cu.
#include "norm_bwd.cuh"

namespace fp8gb {
namespace {

using namespace norms;

// One CTA per SM, of several teams, each with its part of the tokens. Asynchronous bulk copies bring a team's next rows
// into its ring in shared memory while the present one is worked on; w_pre and w_post (times the gate's row where all
// tokens share it) are in shared memory once for all teams. There are dh, dr_out, o, dr and do here, and a norm before
// the next block. SUM: sum dh and sum g are wanted. 16384 x 4096 bf16 with the residual scale's gradient (939 MB): 146 us
// and 6 for the sums, 0.9 of a plain copy's rate (two CTAs per SM with the parameters from L1: 165 in all); 4100 x 1536,
// fp32 stream, layer norms with biases: 28 and 6, where a part's 9 rows are a chain of latencies. Room for 768 threads
// instead of 640 (80 registers) spilled: 42 us for both. SUM with 16 columns a thread spills too (122 to 270 bytes: four
// sums beside three rows): 16384 x 4096 bf16, layer norms, biases, a gate per 512 rows: 211 us, where the rows' bytes take 119.
template <typename TS, typename TB, int E, bool FULL, bool SUM>
__global__ void __launch_bounds__(E == 8 ? 640 : 512, 1)
    norm_bwd_ring_kernel(const NormFwd f, const NormBwd b, float* part, double* part_alpha, int64_t rows_per, int parts, int stages) {
  using R = Row<4, E, FULL>;
  constexpr int H = E / 2, WARPS = E == 8 ? 8 : 16;  // of a team, at most
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Red reds[kMostTeams];
  __shared__ double red_alpha[kMostTeams][16];
  __shared__ __align__(8) uint64_t bars[kMostTeams][kMaxStages];
  __shared__ volatile int fail[kMostTeams][2];  // rows in turn, so that no wait of the next row is taken for this one's
  const int team = threadIdx.y, teams = blockDim.y, p = blockIdx.x * teams + team;
  const int D = static_cast<int>(f.width), c = R::first(threadIdx.x >> 5, threadIdx.x & 31), left = D - c;
  const uint32_t nb = D * sizeof(TB), ns = D * sizeof(TS), bytes = 2 * nb + (b.dres_scale != nullptr ? 3 : 2) * ns;
  const uint32_t at_r_out = nb, at_dr = nb + ns, at_o = nb + 2 * ns, at_r = 2 * nb + 2 * ns;  // after dh
  const uint32_t bar0 = smem_u32(bars[team]), ring0 = team * stages * bytes;
  const int64_t t0 = min(p * rows_per, f.tokens), t1 = min(t0 + rows_per, f.tokens);
  Red& red = reds[team];
  volatile int* failed = fail[team];
  red.clear();
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, 1);
    failed[0] = failed[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto fetch = [&](int64_t t, int s) {  // (a team's thread 0)
    const uint32_t dst = smem_u32(smem) + ring0 + s * bytes, bar = bar0 + 8 * s;
    mbar_arrive_expect_tx(bar, bytes);
    bulk_load(dst, static_cast<const TB*>(b.dh) + t * b.ld_dh, nb, bar);
    bulk_load(dst + at_r_out, static_cast<const TS*>(f.r_out) + t * f.ld_r_out, ns, bar);
    bulk_load(dst + at_dr, static_cast<const TS*>(b.dr_out) + t * b.ld_dr_out, ns, bar);
    bulk_load(dst + at_o, static_cast<const TB*>(f.o) + t * f.ld_o, nb, bar);
    if (b.dres_scale != nullptr) bulk_load(dst + at_r, static_cast<const TS*>(f.r) + t * f.ld_r, ns, bar);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && t0 + s < t1; ++s) fetch(t0 + s, s);
  const bool grouped = f.gate != nullptr && f.gate_rows < f.tokens;
  float* par = reinterpret_cast<float*>(smem + teams * stages * bytes);
  {
    const int tid = team * blockDim.x + threadIdx.x, threads = blockDim.x * teams;
    keep_product(par, f.w_pre, 1.0f, static_cast<const TB*>(nullptr), D, tid, threads);
    keep_product(par + D, f.w_post, 1.0f, grouped ? nullptr : static_cast<const TB*>(f.gate), D, tid, threads);
  }
  __syncthreads();
  const uint32_t w_pre = smem_u32(par + c), w_post = w_pre + 4 * D;
  const float inv = 1.0f / static_cast<float>(D);
  const Pair alpha = both(f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f), zero = both(0.0f);
  Pair aw_pre[H], agz[H], ab_pre[SUM ? H : 1], ag[SUM ? H : 1];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    aw_pre[i] = agz[i] = zero;
    if constexpr (SUM) ab_pre[i] = ag[i] = zero;
  }
  bool spent = false;  // this part's rows of dw_post and db_post hold earlier gates' shares
  // sum g r cancels (its terms have both signs), so the rounding of its running sum is kept: hi + lo
  float al_hi = 0.0f, al_lo = 0.0f;
  float* mine = part + static_cast<int64_t>(p) * kPart * D;
  int64_t grp = 0, grp_end = f.tokens;  // the gate's row, and the first token past its group
  if (f.gate != nullptr) {
    grp = t0 / f.gate_rows;
    grp_end = (grp + 1) * f.gate_rows;
  }
  const int64_t grp0 = grp;
  int turn = 0, stage = 0, odd = 0;
  uint32_t phase = 0;
  bool stop = false;
  for (int64_t t = t0; t < t1; ++t) {
    const float2 pre = __ldg(reinterpret_cast<const float2*>(f.stat_pre) + t);
    const float2 post = f.post != kNone ? __ldg(reinterpret_cast<const float2*>(f.stat_post) + t) : make_float2(0.0f, 1.0f);
    // a wait that ran out is looked at behind a barrier of this row, so that the team stops together
    if (!mbar_wait(bar0 + 8 * stage, phase, f.w, DEV_ERR_WAIT_PRODUCER)) failed[odd] = 1;
    const uint8_t* held = smem + ring0 + stage * bytes;
    if (t == grp_end) {
      ++grp;
      grp_end += f.gate_rows;
    }
    Pair dz[H], z[H], w[H];
    held_row<E, FULL, TB>(held, c, left, dz);
    held_row<E, FULL, TS>(held + at_r_out, c, left, z);
    if constexpr (SUM) {
#pragma unroll
      for (int i = 0; i < H; ++i) ab_pre[i] = add2(ab_pre[i], dz[i]);
    }
    if (f.pre == kLayer) {
      const Pair m = both(-pre.x);
#pragma unroll
      for (int i = 0; i < H; ++i) z[i] = add2(z[i], m);
    }
    {
      const Pair rstd = both(pre.y);
      Pair sq = zero;
      R::load_shared(w_pre, left, w);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        z[i] = mul2(z[i], rstd);
        aw_pre[i] = fma2(dz[i], z[i], aw_pre[i]);
        dz[i] = mul2(dz[i], w[i]);
        sq = fma2(dz[i], z[i], sq);
      }
      Pair m1 = zero;
      float q1;
      if (f.pre == kLayer) {
        Pair sm = zero;
#pragma unroll
        for (int i = 0; i < H; ++i) sm = add2(sm, dz[i]);
        const float2 s = team_sum<WARPS>(make_float2(sum2(sm), sum2(sq)), red, turn);
        m1 = both(-s.x * inv);
        q1 = s.y * inv;
      } else {
        q1 = team_sum<WARPS>(sum2(sq), red, turn) * inv;
      }
      const Pair q = both(-q1);
      held_row<E, FULL, TS>(held + at_dr, c, left, w);
#pragma unroll
      for (int i = 0; i < H; ++i) dz[i] = fma2(z[i], q, dz[i]);
      if (f.pre == kLayer) {
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = add2(dz[i], m1);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) dz[i] = fma2(dz[i], rstd, w[i]);
    }
    // dz: g, the gradient at r'
    R::clear(dz, left);
    if (b.dres_scale != nullptr) {
      held_row<E, FULL, TS>(held + at_r, c, left, z);
      Pair s = zero;
#pragma unroll
      for (int i = 0; i < H; ++i) s = fma2(dz[i], z[i], s);
      const float a = sum2(s), sum = __fadd_rn(al_hi, a), took = __fsub_rn(sum, al_hi);  // two-sum
      al_lo += __fadd_rn(__fsub_rn(al_hi, __fsub_rn(sum, took)), __fsub_rn(a, took));
      al_hi = sum;
    }
#pragma unroll
    for (int i = 0; i < H; ++i) w[i] = mul2(dz[i], alpha);
    R::store(static_cast<TS*>(b.dr) + t * b.ld_dr + c, left, w);
    held_row<E, FULL, TB>(held + at_o, c, left, z);
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
    R::load_shared(w_post, left, w);
    Pair sq = zero;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      agz[i] = fma2(dz[i], z[i], agz[i]);
      if constexpr (SUM) ag[i] = add2(ag[i], dz[i]);
      dz[i] = mul2(dz[i], w[i]);
    }
    if (grouped) {
      R::template load<false>(static_cast<const TB*>(f.gate) + grp * f.ld_gate + c, left, w);
#pragma unroll
      for (int i = 0; i < H; ++i) dz[i] = mul2(dz[i], w[i]);
    }
    Pair m2 = zero;
    float q2 = 0.0f;
    if (f.post != kNone) {
#pragma unroll
      for (int i = 0; i < H; ++i) sq = fma2(dz[i], z[i], sq);
      if (f.post == kLayer) {
        Pair sm = zero;
#pragma unroll
        for (int i = 0; i < H; ++i) sm = add2(sm, dz[i]);
        const float2 s = team_sum<WARPS>(make_float2(sum2(sm), sum2(sq)), red, turn);
        m2 = both(-s.x * inv);
        q2 = s.y * inv;
      } else {
        q2 = team_sum<WARPS>(sum2(sq), red, turn) * inv;
      }
    } else {
      team_sync();
    }
    // a barrier of the team is behind its reads of the row: a later one may land there
    stop = failed[odd] != 0;
    if (stop) break;
    if (threadIdx.x == 0 && t + stages < t1) fetch(t + stages, stage);
    odd ^= 1;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (f.post != kNone) {
      const Pair q = both(-q2), rstd = both(post.y);
      if (f.post == kLayer) {
#pragma unroll
        for (int i = 0; i < H; ++i) dz[i] = add2(dz[i], m2);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) dz[i] = mul2(fma2(z[i], q, dz[i]), rstd);
    }
    R::store(static_cast<TB*>(b.dO) + t * b.ld_do + c, left, dz);
    if (t + 1 == t1 || t + 1 == grp_end) {
      // the sums over the rows of this gate, spent on dgate, dw_post and db_post
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
            R::template load<false>(f.b_post + c, left, w);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = fma2(w[i], ag[i], v[i]);
          }
        }
        leave<4, E, FULL, false>((whole ? b.dgate + grp * D : mine + (grp == grp0 ? 4 : 5) * static_cast<int64_t>(D)) + c, left, v);
      }
      auto spend = [&](int k, Pair(&a)[H]) {  // gate times the sum, onto what earlier gates left
        Pair v[H];
        float* to = mine + k * static_cast<int64_t>(D) + c;
        if (f.gate != nullptr) {
          R::template load<false>(static_cast<const TB*>(f.gate) + grp * f.ld_gate + c, left, v);
#pragma unroll
          for (int i = 0; i < H; ++i) a[i] = mul2(a[i], v[i]);
        }
        if (spent) {
          R::template load<true>(to, left, v);
#pragma unroll
          for (int i = 0; i < H; ++i) a[i] = add2(a[i], v[i]);
        }
        leave<4, E, FULL, true>(to, left, a);
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
  if (stop && threadIdx.x == 0) {  // copies in flight land (microseconds) before the CTA can exit
    const unsigned long long w0 = globaltimer_ns();
    while (globaltimer_ns() - w0 < 200000ull) {
    }
  }
  if (p >= parts) return;  // (the last CTA may have more teams than there are parts; no barrier of the CTA follows)
  if (b.dw_pre != nullptr) leave<4, E, FULL, true>(mine + c, left, aw_pre);
  if constexpr (SUM) leave<4, E, FULL, true>(mine + D + c, left, ab_pre);
  if (b.dres_scale != nullptr) {
    double a = static_cast<double>(al_hi) + static_cast<double>(al_lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if ((threadIdx.x & 31) == 0) red_alpha[team][threadIdx.x >> 5] = a;
    team_sync();
    if (threadIdx.x == 0) {
      for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) a += red_alpha[team][w];
      part_alpha[p] = a;
    }
  }
}

template <typename TS, typename TB, int E, bool FULL, bool SUM>
cudaError_t launch_kernel(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, int teams, int stages, int bytes,
                          cudaStream_t stream) {
  static bool done[64] = {};  // the limit is per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
    e = cudaFuncSetAttribute(norm_bwd_ring_kernel<TS, TB, E, FULL, SUM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_bwd_ring_kernel<TS, TB, E, FULL, SUM>, dim3((pl.parts + teams - 1) / teams), dim3(pl.threads, teams), bytes, stream, f, b, part,
                    part_alpha, pl.rows_per, pl.parts, stages);
}

template <typename TS, typename TB>
cudaError_t ring_as(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, cudaStream_t stream, bool* taken) {
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  if (b.dh == nullptr || b.dr_out == nullptr || b.dr == nullptr || b.dO == nullptr || f.o == nullptr || f.pre == kNone ||
      f.width > 8192 || f.width * bs % 16 != 0 || f.width * ss % 16 != 0 || !rows_aligned(b.dh, f.tokens, b.ld_dh, bs, 16) || !rows_aligned(f.r_out, f.tokens, f.ld_r_out, ss, 16) ||
      !rows_aligned(b.dr_out, f.tokens, b.ld_dr_out, ss, 16) || !rows_aligned(f.o, f.tokens, f.ld_o, bs, 16) ||
      (b.dres_scale != nullptr && !rows_aligned(f.r, f.tokens, f.ld_r, ss, 16)) || !rows_aligned(f.gate, gate_groups(f), f.ld_gate, bs, 4 * bs) ||
      !rows_aligned(b.dr, f.tokens, b.ld_dr, ss, 4 * ss) || !rows_aligned(b.dO, f.tokens, b.ld_do, bs, 4 * bs) || !rows_aligned(f.w_post, 1, 0, 4, 16) ||
      !rows_aligned(f.b_post, 1, 0, 4, 16))
    return cudaSuccess;
  const int teams = pl.per_sm;
  const int64_t row = f.width * (2 * bs + (b.dres_scale != nullptr ? 3 : 2) * ss), params = 8 * f.width, room = (kRingBytes - params) / (row * teams);
  if (room < 1) return cudaSuccess;
  const int stages = static_cast<int>(room < kMaxStages ? room : kMaxStages), bytes = static_cast<int>(params + row * teams * stages);
  const bool sum = sums_wanted(f, b);
  *taken = true;
  if (columns_of(f.width) == 8) {
    if (f.width % 256 == 0)
      return sum ? launch_kernel<TS, TB, 8, true, true>(f, b, pl, part, part_alpha, teams, stages, bytes, stream)
                 : launch_kernel<TS, TB, 8, true, false>(f, b, pl, part, part_alpha, teams, stages, bytes, stream);
    return sum ? launch_kernel<TS, TB, 8, false, true>(f, b, pl, part, part_alpha, teams, stages, bytes, stream)
               : launch_kernel<TS, TB, 8, false, false>(f, b, pl, part, part_alpha, teams, stages, bytes, stream);
  }
  if (f.width % 512 == 0)
    return sum ? launch_kernel<TS, TB, 16, true, true>(f, b, pl, part, part_alpha, teams, stages, bytes, stream)
               : launch_kernel<TS, TB, 16, true, false>(f, b, pl, part, part_alpha, teams, stages, bytes, stream);
  return sum ? launch_kernel<TS, TB, 16, false, true>(f, b, pl, part, part_alpha, teams, stages, bytes, stream)
             : launch_kernel<TS, TB, 16, false, false>(f, b, pl, part, part_alpha, teams, stages, bytes, stream);
}

}  // namespace

cudaError_t launch_norm_bwd_ring(const NormFwd& f, const NormBwd& b, const BwdPlan& pl, float* part, double* part_alpha, cudaStream_t stream,
                                 bool* taken) {
  if (f.stream_f32)
    return f.block_f32 ? ring_as<float, float>(f, b, pl, part, part_alpha, stream, taken) : ring_as<float, bf16>(f, b, pl, part, part_alpha, stream, taken);
  return f.block_f32 ? cudaSuccess : ring_as<bf16, bf16>(f, b, pl, part, part_alpha, stream, taken);
}

}  // namespace fp8gb
