// norm_fwd_ring.cu -- forward of the norms around a block for many rows (HBM-bound: 4 passes over the rows, 8 bytes
// per element in bf16).
#include "norm_emit.cuh"

namespace fp8gb {
namespace {

using namespace norms;

constexpr int kMostTeams = 12;  // rows that a CTA works on at once

// Mean and 1 / root of a team's row.
template <int WARPS, int E, bool FULL>
__device__ __forceinline__ float2 team_stat(int kind, float inv, float eps, const Pair (&v)[E / 2], int left, Red& red, int& turn) {
  float2 st = make_float2(0.0f, 1.0f);
  if (kind == kNone) return st;
  Pair q = both(0.0f);
  if (kind == kLayer) {
    Pair a = both(0.0f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) a = add2(a, v[i]);  // (zero past the row)
    st.x = team_sum<WARPS>(sum2(a), red, turn) * inv;
    const Pair m = both(-st.x);
    Pair z[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) z[i] = add2(v[i], m);
    Row<4, E, FULL>::clear(z, left);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) q = fma2(z[i], z[i], q);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) q = fma2(v[i], v[i], q);
  }
  st.y = inv_sqrt(fmaf(team_sum<WARPS>(sum2(q), red, turn), inv, eps));
  return st;
}

template <int E>
__device__ __forceinline__ void normalize(Pair (&x)[E / 2], int kind, float2 st) {
  if (kind == kLayer) {  // the mean is taken off before the scaling, so that a large one does not cancel
    const Pair m = both(-st.x);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = add2(x[i], m);
  }
  const Pair rstd = both(st.y);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], rstd);
}

// At most one CTA per SM, of several teams of up to WARPS warps that take rows in turn. Asynchronous bulk copies bring a
// team's next rows into its ring in shared memory while the present one is worked on, so the loads never wait for the
// arithmetic; the parameters are in shared memory once for all teams, ones where there are none and the gate's row
// multiplied in where all tokens share it. 16384 x 4096 bf16: parameters read from L1 beside the rings (some 30 KB of it,
// half of the reads missed) 110 us; kept in shared memory 95; with as many teams as the memory needs (ring_plan) 82.7,
// 6.5 TB/s. BIAS: there is a bias.
template <typename TS, typename TB, int E, bool FULL, int WARPS, bool BIAS>
__global__ void __launch_bounds__(WARPS == 16 ? 512 : 768, 1) norm_fwd_ring_kernel(const NormFwd f, uint32_t gate_rows, int stages) {
  using R = Row<4, E, FULL>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Red reds[kMostTeams];
  __shared__ float table[8];
  __shared__ __align__(8) uint64_t bars[kMostTeams][kMaxStages];
  __shared__ volatile int fail[kMostTeams][2];  // rows in turn, so that no wait of the next row is taken for this one's
  const int team = threadIdx.y, teams = blockDim.y;
  const int D = static_cast<int>(f.width), c = R::first(threadIdx.x >> 5, threadIdx.x & 31), left = D - c;
  const uint32_t r_bytes = D * sizeof(TS), o_bytes = D * sizeof(TB), bytes = r_bytes + o_bytes;
  const uint32_t bar0 = smem_u32(bars[team]), ring0 = team * stages * bytes;
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
  auto fetch = [&](uint32_t t, int s) {  // (a team's thread 0)
    const uint32_t dst = smem_u32(smem) + ring0 + s * bytes;
    mbar_arrive_expect_tx(bar0 + 8 * s, bytes);
    bulk_load(dst, static_cast<const TS*>(f.r) + t * f.ld_r, r_bytes, bar0 + 8 * s);
    bulk_load(dst + r_bytes, static_cast<const TB*>(f.o) + t * f.ld_o, o_bytes, bar0 + 8 * s);
  };
  const uint32_t T = static_cast<uint32_t>(f.tokens), t0 = blockIdx.x * teams + team, step = gridDim.x * teams;
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && t0 + s * static_cast<uint64_t>(step) < T; ++s) fetch(t0 + s * step, s);
  const int tid = team * blockDim.x + threadIdx.x, threads = blockDim.x * teams;
  const TB* gate = static_cast<const TB*>(f.gate);
  const bool grouped = gate != nullptr && gate_rows < T;
  float* par = reinterpret_cast<float*>(smem + teams * stages * bytes);  // w_post, w_pre, b_post, b_pre
  {
    const TB* one = grouped ? nullptr : gate;
    keep_product(par, f.w_post, 1.0f, one, D, tid, threads);
    keep_product(par + D, f.w_pre, 1.0f, static_cast<const TB*>(nullptr), D, tid, threads);
    if constexpr (BIAS) {
      keep_product(par + 2 * D, f.b_post, 0.0f, f.b_post != nullptr ? one : nullptr, D, tid, threads);  // (no bias: 0, not 0 times the gate)
      keep_product(par + 3 * D, f.b_pre, 0.0f, static_cast<const TB*>(nullptr), D, tid, threads);
    }
  }
  fill_table(f, table, tid);
  if (f.hq != nullptr) fill_scales(f, blockIdx.x * static_cast<int64_t>(threads) + tid, static_cast<int64_t>(gridDim.x) * threads);
  __syncthreads();
  const uint32_t w_post = smem_u32(par + c), w_pre = w_post + 4 * D, b_post = w_pre + 4 * D, b_pre = b_post + 4 * D;
  const Pair alpha = both(f.res_scale != nullptr ? __ldg(f.res_scale) : 1.0f);
  const float inv = 1.0f / static_cast<float>(D);
  int turn = 0, stage = 0, odd = 0;
  uint32_t phase = 0;
  bool stop = false;
  for (uint64_t row = t0; row < T; row += step) {
    const uint32_t t = static_cast<uint32_t>(row);
    // a wait that ran out is looked at behind this row's barrier, so that the team stops together
    if (!mbar_wait(bar0 + 8 * stage, phase, f.w, DEV_ERR_WAIT_PRODUCER)) failed[odd] = 1;
    const uint8_t* held = smem + ring0 + stage * bytes;
    Pair x[E / 2], n[E / 2];
    held_row<E, FULL, TS>(held, c, left, x);
    held_row<E, FULL, TB>(held + r_bytes, c, left, n);
    const float2 post = team_stat<WARPS, E, FULL>(f.post, inv, f.eps, n, left, red, turn);
    if (f.post == kNone) team_sync();
    // a barrier of the team is behind its reads of the row: a later one may land there
    stop = failed[odd] != 0;
    if (stop) break;
    if (threadIdx.x == 0) {
      const uint64_t next = row + static_cast<uint64_t>(stages) * step;
      if (next < T) fetch(static_cast<uint32_t>(next), stage);
      if (f.stat_post != nullptr) reinterpret_cast<float2*>(f.stat_post)[t] = post;
    }
    odd ^= 1;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    normalize<E>(n, f.post, post);
    Pair p[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], alpha);
    R::load_shared(w_post, left, p);
    if (grouped) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) n[i] = mul2(n[i], p[i]);
      if constexpr (BIAS) {
        R::load_shared(b_post, left, p);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) n[i] = add2(n[i], p[i]);
      }
      R::template load<false>(gate + (t / gate_rows) * f.ld_gate + c, left, p);
    } else if constexpr (BIAS) {
      Pair q[E / 2];
      R::load_shared(b_post, left, q);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = add2(x[i], q[i]);
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = fma2(n[i], p[i], x[i]);
    R::clear(x, left);  // (past the row: what the norm made of nothing)
    if (f.r_out != nullptr) R::store(static_cast<TS*>(f.r_out) + t * f.ld_r_out + c, left, x);
    const float2 pre = team_stat<WARPS, E, FULL>(f.pre, inv, f.eps, x, left, red, turn);
    if (threadIdx.x == 0 && f.stat_pre != nullptr) reinterpret_cast<float2*>(f.stat_pre)[t] = pre;
    normalize<E>(x, f.pre, pre);
    R::load_shared(w_pre, left, p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], p[i]);
    if constexpr (BIAS) {
      R::load_shared(b_pre, left, p);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = add2(x[i], p[i]);
    }
    if (f.h != nullptr) R::store(static_cast<TB*>(f.h) + t * f.ld_h + c, left, x);
    if (f.hq != nullptr) {
      if (f.h_fmt == 0)
        emit_row<0, 4, E>(f, x, t, c, left, table);
      else
        emit_row<1, 4, E>(f, x, t, c, left, table);
    }
  }
  if (stop && threadIdx.x == 0) {  // copies in flight land (microseconds) before the CTA can exit
    const unsigned long long w0 = globaltimer_ns();
    while (globaltimer_ns() - w0 < 200000ull) {
    }
  }
}

struct RingPlan {
  int threads, teams, ctas, stages, bytes;  // of a team, teams, CTAs, rows each team holds, shared memory
};

// As many rows at once as keep the memory busy, and no more: the teams' time for a row, which grows with the warps on an SM,
// times the memory's rate over the row's bytes. Past that the copies and stores only stand in each other's way:
// 16384 x 4096 bf16 in 3 teams on each of 152 SMs 95 us, in 2 on 143 of them 82.7 (6.5 TB/s), in 2 on 128 90.6; 32768 x 2048
// 94 and 82; 16384 x 4096 with an fp32 stream 136 in 3 teams, 129 in 1. The constants are measured times (us) of a row alone: two
// layer norms 1.7, two root mean squares 0.88, one norm 0.55, with 4-bit codes 0.5 more, above 8 warps 0.2 more.
RingPlan ring_plan(const NormFwd& f, int64_t row, int columns, bool bias) {
  RingPlan p{};
  p.threads = static_cast<int>((f.width + 32 * columns - 1) / (32 * columns)) * 32;
  const int sms = num_sms(), warps = p.threads / 32, room_for = p.threads > 384 ? 1 : 768 / p.threads, most = room_for < kMostTeams ? room_for : kMostTeams;
  const int64_t ss = f.stream_f32 ? 4 : 2, bs = f.block_f32 ? 4 : 2;
  const float bytes = static_cast<float>(f.width) *
                      (static_cast<float>(ss + bs + (f.r_out != nullptr ? ss : 0) + (f.h != nullptr ? bs : 0)) + (f.hq != nullptr ? 0.5625f : 0.0f));
  float chain = f.post == kLayer || f.pre == kLayer ? 1.7f : f.post == kNone || f.pre == kNone ? 0.55f : 0.88f;
  if (warps > 8) chain += 0.2f;
  if (f.hq != nullptr) chain += 0.5f;
  float rows = 0.0f;
  for (p.teams = 1;; ++p.teams) {
    rows = (chain + 0.034f * static_cast<float>(p.teams * warps)) * 6.6e6f / bytes;
    if (p.teams == most || static_cast<float>(p.teams * sms) >= 0.98f * rows) break;
  }
  const int ctas = static_cast<int>(rows / static_cast<float>(p.teams)) + 1;
  p.ctas = ctas < sms ? ctas : sms;
  const int64_t params = (bias ? 16 : 8) * f.width, room = (kRingBytes - params) / (row * p.teams);
  p.stages = static_cast<int>(room < 0 ? 0 : room < kMaxStages ? room : kMaxStages);
  p.bytes = static_cast<int>(params + p.stages * p.teams * row);
  return p;
}

template <typename TS, typename TB, int E, bool FULL, int WARPS, bool BIAS>
cudaError_t launch_kernel(const NormFwd& f, const RingPlan& p, cudaStream_t stream) {
  static bool done[64] = {};  // the limit is per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
    e = cudaFuncSetAttribute(norm_fwd_ring_kernel<TS, TB, E, FULL, WARPS, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return e;
  NormFwd g = f;
  g.w = wait_ctl();
  if (g.w.err == nullptr) return cudaErrorInvalidDevice;
  return launch_pdl(norm_fwd_ring_kernel<TS, TB, E, FULL, WARPS, BIAS>, dim3(p.ctas), dim3(p.threads, p.teams), p.bytes, stream, g, gate_rows_of(f), p.stages);
}

template <typename TS, typename TB>
cudaError_t ring_as(const NormFwd& f, cudaStream_t stream, bool* taken) {
  const int64_t ss = sizeof(TS), bs = sizeof(TB);
  // The parameters and the first rows have to come in before any work: it takes some rows per SM to pay (us here, and a row
  // per CTA from registers: 1000 x 4096 8.6, 7.7; 2000 x 4096 15.3, 17.1; 1000 x 8192 17.5, 18.8; 400 x 768 4.0, 3.4; 16384 x 768
  // 22.4, 27.9; 60000 x 512 44, 44)
  const int64_t rows = f.width > 4096 ? 4 : f.width >= 1024 ? 8 : 32;
  if (f.o == nullptr || f.tokens < rows * num_sms() || f.width <= 512 || f.width > 8192 || f.width * ss % 16 != 0 || f.width * bs % 16 != 0 || !rows_aligned(f.r, f.tokens, f.ld_r, ss, 16) ||
      !rows_aligned(f.o, f.tokens, f.ld_o, bs, 16) || !rows_aligned(f.r_out, f.tokens, f.ld_r_out, ss, 4 * ss) || !rows_aligned(f.h, f.tokens, f.ld_h, bs, 4 * bs) ||
      !rows_aligned(f.gate, gate_groups(f), f.ld_gate, bs, 4 * bs))
    return cudaSuccess;
  const bool bias = f.b_post != nullptr || f.b_pre != nullptr, full = f.width % 512 == 0;
  const RingPlan p = ring_plan(f, f.width * (ss + bs), 16, bias);
  if (p.stages == 0) return cudaSuccess;
  *taken = true;
  // (8 warps are sums of two reads: with 12 for all of them two layer norms took 117 us instead of 106)
  if (p.threads <= 256) {
    if (full) return bias ? launch_kernel<TS, TB, 16, true, 8, true>(f, p, stream) : launch_kernel<TS, TB, 16, true, 8, false>(f, p, stream);
    return bias ? launch_kernel<TS, TB, 16, false, 8, true>(f, p, stream) : launch_kernel<TS, TB, 16, false, 8, false>(f, p, stream);
  }
  if (p.threads <= 384) return bias ? launch_kernel<TS, TB, 16, false, 12, true>(f, p, stream) : launch_kernel<TS, TB, 16, false, 12, false>(f, p, stream);
  if (full) return bias ? launch_kernel<TS, TB, 16, true, 16, true>(f, p, stream) : launch_kernel<TS, TB, 16, true, 16, false>(f, p, stream);
  return bias ? launch_kernel<TS, TB, 16, false, 16, true>(f, p, stream) : launch_kernel<TS, TB, 16, false, 16, false>(f, p, stream);
}

}  // namespace

cudaError_t launch_norm_fwd_ring(const NormFwd& f, cudaStream_t stream, bool* taken) {
  if (f.stream_f32)
    return f.block_f32 ? ring_as<float, float>(f, stream, taken) : ring_as<float, bf16>(f, stream, taken);
  return f.block_f32 ? cudaSuccess : ring_as<bf16, bf16>(f, stream, taken);
}

}  // namespace fp8gb
