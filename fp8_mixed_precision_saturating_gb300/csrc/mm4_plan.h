// mm4_plan.h -- how a product of 4-bit operands is run, from its sizes and what the device holds (host code).
#pragma once
#include <cstdint>

namespace fp8gb {

constexpr int kMm4StageK = 256;     // contraction elements per stage
constexpr int kMm4PairSplits = 4;   // parts of K over the CTA pairs of a cluster, at most
constexpr int kMm4Splits = 8;       // over the CTAs of a cluster

// CTA pairs (bn == 0), or clusters of `splits` single CTAs with tiles of 128 x bn; splits == 0: the device holds none.
struct Mm4Plan {
  int bn, splits;
};

// How many clusters of each number of splits the device holds at once (0: not one); CTA pairs, and single CTAs with
// 128-wide tiles.
struct Mm4Clusters {
  int pair[kMm4PairSplits + 1], one[kMm4Splits + 1];
};

// Up to 64 rows of A the weights' bytes and the latency decide: one CTA per SM (more of them measured slower:
// 1 x 4096 x 4096 took 3.9 us in 128 CTAs, 4.4 in 256), at least two stages each.
inline Mm4Plan mm4_plan_few_rows(int64_t M, int64_t N, int64_t K, int64_t sms) {
  const int64_t stages = (K + kMm4StageK - 1) / kMm4StageK;
  int64_t s = sms / ((N + 127) / 128);
  s = s < stages / 2 ? s : stages / 2;
  return {M <= 16 ? 16 : M <= 32 ? 32 : 64, static_cast<int>(s < 1 ? 1 : s > kMm4Splits ? kMm4Splits : s)};
}

// The cheapest plan above 64 rows of A, by the measured times of a stage and of what comes before and after the stages
// (us, GB300): a pair does 256 x 256 x 256 in 0.27, a CTA 128 x 128 x 256 in 0.31; summing the parts of a split tile takes
// 3.6 on pairs (128 KB per CTA), 1.2 otherwise, where the single CTA's unsplit epilogue takes 2. Clusters that the device
// does not hold (a context on part of the SMs may have none of the large ones) are not offered.
inline Mm4Plan mm4_plan(int64_t M, int64_t N, int64_t K, int64_t sms, const Mm4Clusters& fit) {
  const int64_t stages = (K + kMm4StageK - 1) / kMm4StageK;
  Mm4Plan plan = {0, 0};
  float best = 0.0f;
  auto offer = [&](int bn, int splits, float us) {
    if (plan.splits != 0 && us >= best) return;
    best = us;
    plan = {bn, splits};
  };
  const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256), small = (M + 127) / 128 * ((N + 127) / 128);
  for (int s = 1; s <= kMm4PairSplits && s <= stages; ++s)
    if (fit.pair[s] > 0 && (s == 1 || tiles <= fit.pair[s]))
      offer(0, s, 4.3f + 0.27f * static_cast<float>((stages + s - 1) / s * ((tiles + fit.pair[s] - 1) / fit.pair[s])) + (s > 1 ? 3.6f : 0.0f));
  for (int s = 1; s <= kMm4Splits && s <= stages; ++s)
    if (fit.one[s] > 0 && small <= (s == 1 ? sms : fit.one[s]))
      offer(128, s, 4.0f + 0.31f * static_cast<float>((stages + s - 1) / s) + (s > 1 ? 1.2f : 2.0f));
  return plan;
}

}  // namespace fp8gb
