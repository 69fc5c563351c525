// norm_bwd.cuh -- what the backward kernels of the norms share beyond norm.cuh: how the tokens are split and where the
// parts' column sums go.
#pragma once
#include "norm.cuh"

namespace fp8gb {
namespace norms {

// Part p of the tokens is [p R, (p + 1) R); the CTA (or team) that takes it leaves its share of every column sum in
// its own rows of the workspace: 4 rows for the parameters, then 2 for the gate gradient of the
// groups that it shares with its neighbours (its first group, its last). A group inside one part is
// written out by its CTA alone. A second kernel adds the shares up in order.
constexpr int kPart = 6;

// The split of the tokens, from the sizes alone: parts of consecutive rows, each worked on by `threads` threads that
// hold columns_of(width) columns each, as many per SM as the registers allow (some 100 a thread with 8 columns, 128
// with 16).
struct BwdPlan {
  int parts, threads, per_sm;
  int64_t rows_per;
};

constexpr int kMostTeams = 15;  // (a CTA of several parts keeps a named barrier for each, besides its own)

// 8 columns a thread make more warps of a row (4100 x 1536, layer norms with a gate: 33.9 us, with 16 columns 42.7); rows
// that are no whole items of 4 are read in single elements, where the loads of 16 columns in flight count for more
// (4099 x 1537 bf16: 47.0 us, with 8 columns 54.4)
inline int columns_of(int64_t width) { return width <= (width % 4 == 0 ? 2048 : 1024) ? 8 : 16; }

inline BwdPlan bwd_plan(int64_t tokens, int64_t width) {
  BwdPlan p;
  const int64_t per = 32 * columns_of(width);
  p.threads = width <= 8192 ? static_cast<int>((width + per - 1) / per) * 32 : kThreads;
  p.per_sm = (columns_of(width) == 8 ? 640 : 512) / p.threads;
  p.per_sm = p.per_sm < 1 ? 1 : p.per_sm > kMostTeams ? kMostTeams : p.per_sm;
  const int64_t most = static_cast<int64_t>(p.per_sm) * num_sms();
  p.rows_per = (tokens + most - 1) / most;
  p.parts = static_cast<int>((tokens + p.rows_per - 1) / p.rows_per);
  return p;
}

// Whether sum dh and sum g are needed: a bias's gradient, or the gate's where there is a bias.
inline bool sums_wanted(const NormFwd& f, const NormBwd& b) {
  return b.db_pre != nullptr || b.db_post != nullptr || (b.dgate != nullptr && f.b_post != nullptr);
}

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

}  // namespace norms

// Rows of whole 16 bytes with every gradient of a training step (norm_bwd_ring.cu); taken: whether it was one for that
// kernel.
cudaError_t launch_norm_bwd_ring(const NormFwd& f, const NormBwd& b, const norms::BwdPlan& pl, float* part, double* part_alpha, cudaStream_t stream,
                                 bool* taken);

}  // namespace fp8gb
