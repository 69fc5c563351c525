// gemm4.cu -- C = A B^T of two microscaled 4-bit operands on the tensor cores (tcgen05, kind::mxf4nvf4 and
// kind::mxf4, fp32 accumulation).
//
// Formats and layout: include/fp8gb.h, "Microscaled 4-bit operands".
//   C[m, n] = round( d_a d_b sum_g c_a[m, g] c_b[n, g] sum_{k in g} a[m, k] b[n, k] )
//
// The tensor cores take the codes as stored (two per byte, 128-byte-swizzled rows of 256 K) and apply the
// group scales themselves, from tensor memory. A stage of either kernel holds 256 K of its rows and the
// scale atoms of those K (4 atoms per 128 rows for NVFP4, 2 for MXFP4); K past the operand's end arrives as
// zero codes (TMA fill) under zero or tiny scales, so no size of K needs a branch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "fp4.cuh"
#include "kernels.h"
#include "mm4_plan.h"
#include "ptx.cuh"

namespace fp8gb {
namespace {

constexpr int kStageK = kMm4StageK;     // contraction elements per stage: rows of 128 bytes
constexpr int kOpBytes = 128 * 128;     // 128 rows of an operand
constexpr int kStg = 32 * 128;          // an epilogue warp's staging buffer: 32 rows of 128 bytes

template <int FMT>
constexpr int kAtoms = FMT == 0 ? 4 : 2;  // scale atoms per 128 rows and stage

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

// The scale and MMA instructions of one stage. Operand tiles at sa, sb; their scale atoms at fa ([atom][512]) and
// fb ([128-row block][atom][512]); scale columns at ca (4 per atom) and cb (4 NB per atom).
template <int FMT, bool PAIR, int NB>
__device__ __forceinline__ void stage_mma(uint32_t d, uint32_t sa, uint32_t sb, uint32_t fa, uint32_t fb, uint32_t ca, uint32_t cb,
                                          uint32_t idesc, bool first) {
  constexpr int KA = kAtoms<FMT>;
  auto copy = [](uint32_t col, uint32_t at) {
    if constexpr (PAIR)
      tmem_cp_32x128b_x4_pair(col, smem_desc_plain128(at));
    else
      tmem_cp_32x128b_x4(col, smem_desc_plain128(at));
  };
#pragma unroll
  for (int j = 0; j < KA; ++j) {
    copy(ca + 4 * j, fa + 512 * j);
#pragma unroll
    for (int b = 0; b < NB; ++b) copy(cb + 4 * (NB * j + b), fb + 512 * (KA * b + j));
  }
  const uint64_t adesc = smem_desc_sw128(sa), bdesc = smem_desc_sw128(sb);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = FMT == 0 ? k : k >> 1;
    const uint32_t ids = FMT == 0 ? 0u : idesc_sf_ids(2 * (k & 1), 2 * (k & 1));
    mma_f4<FMT, PAIR>(d, adesc + 2 * k, bdesc + 2 * k, idesc | ids, ca + 4 * j, cb + 4 * NB * j, !(first && k == 0));
  }
}

__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cta.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Every thread's share of a reduction over the CTAs first, first + step, ... (n of them, at most MOST) of the cluster:
// items begin, begin + stride, ... below end, four fp32 values each at at(item) in every CTA's shared memory, summed in
// CTA order and handed to out(item, sum). The loads of U items are in flight together, and this CTA's own values (its
// place among the n is `own`) are read as local ones: two pairs' 128 x 256 tiles took 3.1 us when they went the
// remote way too.
template <int MOST, int U, typename At, typename Out>
__device__ __forceinline__ void cluster_sum(int begin, int end, int stride, int first, int step, int n, int own, At at, Out out) {
  for (int i = begin; i < end; i += U * stride) {
    float4 v[U][MOST];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < MOST; ++r)
        if (r < n && i + u * stride < end)
          v[u][r] = r == own ? ld_shared_f32x4(at(i + u * stride)) : ld_cluster_f32x4(mapa_shared(at(i + u * stride), static_cast<uint32_t>(first + r * step)));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float4 s = v[u][0];
#pragma unroll
      for (int r = 1; r < MOST; ++r)
        if (r < n) s = make_float4(__fadd_rn(s.x, v[u][r].x), __fadd_rn(s.y, v[u][r].y), __fadd_rn(s.z, v[u][r].z), __fadd_rn(s.w, v[u][r].w));
      if (i + u * stride < end) out(i + u * stride, s);
    }
  }
}

// Four neighbouring results times d, `left` of them inside the row (rows and columns in fours are aligned).
template <typename T>
__device__ __forceinline__ void put4(T* p, float4 s, float d, int left) {
  const float v[4] = {__fmul_rn(s.x, d), __fmul_rn(s.y, d), __fmul_rn(s.z, d), __fmul_rn(s.w, d)};
  if (left >= 4) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    else
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < left) {
        if constexpr (sizeof(T) == 2)
          p[j] = __float2bfloat16_rn(v[j]);
        else
          p[j] = v[j];
      }
  }
}

template <typename T>
__device__ __forceinline__ void put(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = __float2bfloat16_rn(v);
  else
    *p = v;
}

// ---------------------------------------------------------------------------------------
// Many rows: persistent CTA pairs, tiles of 256 x 256
// ---------------------------------------------------------------------------------------
// Each CTA of a pair loads its 128 rows of A, half of B's 256 rows, its rows' scales and all of B's (its
// tensor core computes every column). Two accumulators of 256 columns and the scale columns do not fit in
// 512, so the second accumulator starts before the first one ends: the next tile's MMAs may begin once the
// columns that the two share have been read, which the epilogue does first.
// With too few tiles for the GPU, the pairs of a larger cluster take consecutive ranges of one tile's K (SPLIT): each
// CTA writes its 128 x 256 fp32 partial tile where its operands were, and then sums a share of the rows over the
// pairs, in order, and stores it (the same bits every time; no workspace, no atomics).
// 16384 x 14336 x 4096, NVFP4 to bf16: 285 us (6.8 PFLOP/s; 314 where the power limit holds the clock down), bound by the tensor
// pipe, active 73 % of the time; with a lane index instead of an elected lane issuing it took 511. 1536 x 1000 x 16379: 24
// tiles, K in 2: 18 us (on single CTAs 24.6), of which the sum is 3.6.
template <int FMT>
struct Pair {
  static constexpr int KA = kAtoms<FMT>;
  static constexpr int SF_BYTES = 512 * 3 * KA;
  static constexpr int TX_BYTES = 2 * kOpBytes + SF_BYTES;  // per CTA and stage
  static constexpr int STAGES = 5;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int SFA = 512 - 12 * KA, SFB = SFA + 4 * KA;  // scale columns
  static constexpr int ACC1 = SFA - 256;                         // first column of the second accumulator
  static constexpr int OFF_SF = STAGES * 2 * kOpBytes;
  static constexpr int OFF_STG = OFF_SF + STAGES * SF_BYTES;
  static constexpr int OFF_BAR = OFF_STG + EPI_WARPS * kStg;
  // SPLIT: the partial tile lies where the operands were
  static constexpr int TILE_PITCH = 260 * 4;  // bytes of a row: lanes' 16 bytes in different banks
  static_assert(128 * TILE_PITCH <= OFF_SF, "partial tile");
  static constexpr int MOST_SPLITS = kMm4PairSplits;
  static constexpr int NBAR = 2 * STAGES + 4;  // full, empty, tile done [2], shared columns read, final
  static constexpr int OFF_SLOT = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM = OFF_SLOT + 16 + 1024;
  static_assert(OFF_STG % 1024 == 0 && SMEM <= 232448, "shared memory");
  // the shared columns lie in the first accumulator's last 64 and the second's first 64
  static_assert(ACC1 >= 192, "shared columns");
};

struct PairParams {
  int M, N, tiles, num_m, num_n, stages_k, group_m, splits;
  void* C;
  int64_t ldc;
  const float* da;
  const float* db;
  WaitCtl w;
};

// Tile t: groups of group_m row blocks sweep the column blocks together, so that a group's tiles read B from L2.
__device__ __forceinline__ void tile_at(int t, const PairParams& p, int& mb, int& nb) {
  const int per = p.group_m * p.num_n, g = t / per, rows = min(p.group_m, p.num_m - g * p.group_m), l = t - g * per;
  nb = l / rows;
  mb = g * p.group_m + (l - nb * rows);
}

template <int FMT, bool F32, bool SPLIT>
__global__ void __launch_bounds__(Pair<FMT>::THREADS, 1)
    mm4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmSA,
                    const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmC, const __grid_constant__ PairParams p) {
  using C = Pair<FMT>;
  using T = std::conditional_t<F32, float, __nv_bfloat16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar_full = base + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES, bar_done = bar_empty + 8 * C::STAGES;
  const uint32_t bar_free = bar_done + 16, bar_final = bar_free + 8;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  // SPLIT: pair `part` of the cluster's `splits` takes K stages [k0, k1) of the cluster's one tile
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
  const int part = static_cast<int>(crank >> 1);
  const int first = SPLIT ? blockIdx.x / (2 * p.splits) : blockIdx.x >> 1, step = SPLIT ? p.tiles : gridDim.x >> 1;
  const int k0 = SPLIT ? p.stages_k * part / p.splits : 0, k1 = SPLIT ? p.stages_k * (part + 1) / p.splits : p.stages_k;
  const uint16_t pair_mask = static_cast<uint16_t>(0x3u << lead);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_done, 1);
    mbar_init(bar_done + 8, 1);
    mbar_init(bar_free, 2 * C::EPI_WARPS);
    mbar_init(bar_final, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t full_lead = mapa_shared(bar_full, lead);
    for (int t = first; ok && t < p.tiles; t += step) {
      int mb, nb;
      tile_at(t, p, mb, nb);
      for (int k = k0; k < k1; ++k) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_empty + 8 * stage, phase ^ 1u, p.w, DEV_ERR_WAIT_PRODUCER));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t sa = base + stage * 2 * kOpBytes, sf = base + C::OFF_SF + stage * C::SF_BYTES, fb = full_lead + 8 * stage;
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * C::TX_BYTES);  // both CTAs' bytes
          tma_load_2d_pair(sa, &tmA, fb, k * 128, mb * 256 + static_cast<int>(rank) * 128);
          tma_load_2d_pair(sa + kOpBytes, &tmB, fb, k * 128, nb * 256 + static_cast<int>(rank) * 128);
          tma_load_3d_pair(sf, &tmSA, fb, 0, k * C::KA, mb * 2 + static_cast<int>(rank));
          tma_load_3d_pair(sf + 512 * C::KA, &tmSB, fb, 0, k * C::KA, nb * 2);
        }
        __syncwarp();
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {  // let the loads in flight land (microseconds) before the CTA can exit
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {  // the whole warp walks the stages, one lane issues
      const uint32_t idesc = idesc_f4(FMT, 256, 256);
      int stage = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; ok && t < p.tiles; t += step, ++i) {
        // the tile before has been read as far as the two accumulators share columns (and the one before it, whose
        // accumulator this is, altogether)
        ok = i == 0 || mbar_wait(bar_free, (i - 1) & 1, p.w, DEV_ERR_WAIT_MMA);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const uint32_t d = tmem + (i & 1 ? C::ACC1 : 0);
        for (int k = k0; ok && k < k1; ++k) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * stage, phase, p.w, DEV_ERR_WAIT_MMA));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = base + stage * 2 * kOpBytes, sf = base + C::OFF_SF + stage * C::SF_BYTES;
            stage_mma<FMT, true, 2>(d, sa, sa + kOpBytes, sf, sf + 512 * C::KA, tmem + C::SFA, tmem + C::SFB, idesc, k == k0);
            mma_commit_pair(bar_empty + 8 * stage, pair_mask);
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && elect_one()) mma_commit_pair(bar_done + 8 * (i & 1), pair_mask);
        __syncwarp();
      }
      if (elect_one()) mma_commit_pair(bar_final, static_cast<uint16_t>(1u << lead));
      __syncwarp();
      if (!wait_drain(bar_final, 0, 1000000000ull)) atomicOr(p.w.err, DEV_ERR_WAIT_TEARDOWN);
    }
  } else if constexpr (SPLIT) {
    // this CTA's partial tile: rows of 256 fp32 (every load has landed and every MMA is done)
    const int q = warp & 3, half = (warp - 2) >> 2;
    const bool good = mbar_wait(bar_done, 0, p.w, DEV_ERR_WAIT_EPILOGUE);
    __syncwarp();
    tc_fence_after();
    if (good) {
      uint8_t* row = smem + (q * 32 + lane) * C::TILE_PITCH + half * 512;
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t r[32];
        tmem_ld32(acc + c, r);
        tmem_ld_wait();
        reg_fence(r);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(row + 4 * c + 16 * j) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
      }
      tc_fence_before();
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, q = warp & 3, half = ew >> 2;
    uint8_t* stg = smem + C::OFF_STG + ew * kStg;
    const float d = __fmul_rn(p.da != nullptr ? __ldg(p.da) : 1.0f, p.db != nullptr ? __ldg(p.db) : 1.0f);
    const uint32_t free_lead = mapa_shared(bar_free, lead);
    int i = 0;
    for (int t = first; t < p.tiles; t += step, ++i) {
      int mb, nb;
      tile_at(t, p, mb, nb);
      if (!mbar_wait(bar_done + 8 * (i & 1), (i >> 1) & 1, p.w, DEV_ERR_WAIT_EPILOGUE)) break;
      __syncwarp();
      tc_fence_after();
      const int row0 = mb * 256 + static_cast<int>(rank) * 128 + q * 32;
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (i & 1 ? C::ACC1 : 0);
      // the two warps of a lane quarter take 64-column chunks {0, 2} and {1, 3}; the one that holds the shared
      // columns (chunk 3 of the first accumulator, chunk 0 of the second) reads those first
      const bool holds = half == 1 - (i & 1);
      if (!holds && lane == 0) mbar_arrive_cluster(free_lead);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const int chunk = half + 2 * (half == 1 ? 1 - c : c);
        uint32_t r[64];
        tmem_ld64(acc + chunk * 64, r);
        tmem_ld_wait();
        reg_fence(r);
        if (c == 0 && holds) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(free_lead);
        }
        const int chunk0 = nb * 256 + chunk * 64;
        if (chunk0 + 64 > p.N && (p.N & (F32 ? 3 : 7)) != 0) {
          // the row's end inside 16 bytes: a tiled store would write zeros up to the end of those, so plain stores
          if (row0 + lane < p.M) {
            T* out = static_cast<T*>(p.C) + (row0 + lane) * p.ldc + chunk0;
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (chunk0 + j < p.N) put(out + j, __fmul_rn(__uint_as_float(r[j]), d));
          }
          __syncwarp();
          continue;
        }
        constexpr int PARTS = F32 ? 2 : 1;  // 128 bytes of a row per store: 64 bf16 or 32 fp32
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
          if (lane == 0) bulk_wait_group_read<0>();  // the store before has read the buffer
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 v;
            if constexpr (F32) {
              const int o = 32 * h + 4 * j;
              v = make_uint4(__float_as_uint(__fmul_rn(__uint_as_float(r[o]), d)), __float_as_uint(__fmul_rn(__uint_as_float(r[o + 1]), d)),
                             __float_as_uint(__fmul_rn(__uint_as_float(r[o + 2]), d)), __float_as_uint(__fmul_rn(__uint_as_float(r[o + 3]), d)));
            } else {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2(__fmul_rn(__uint_as_float(r[8 * j + 2 * e]), d), __fmul_rn(__uint_as_float(r[8 * j + 2 * e + 1]), d));
              v = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) * 16)) = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          const int col0 = chunk0 + 32 * h;
          if (lane == 0 && row0 < p.M && col0 < p.N) {  // (the rest is clipped at M and N)
            tma_store_2d(&tmC, smem_u32(stg), col0, row0);
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
    }
    if (lane == 0) bulk_wait_group<0>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no commit or load of the pair targets a CTA that has left; SPLIT: the partial tiles are there
  if constexpr (SPLIT) {
    const float d = __fmul_rn(p.da != nullptr ? __ldg(p.da) : 1.0f, p.db != nullptr ? __ldg(p.db) : 1.0f);
    int mb, nb;
    tile_at(first, p, mb, nb);
    const int row0 = mb * 256 + static_cast<int>(rank) * 128, live = max(0, min(128, p.M - row0));
    const int r0 = live * part / p.splits, r1 = live * (part + 1) / p.splits;
    cluster_sum<C::MOST_SPLITS, 4>(r0 * 64 + static_cast<int>(threadIdx.x), r1 * 64, C::THREADS, static_cast<int>(rank), 2, p.splits, part,
                                   [&](int i) { return base + (i >> 6) * C::TILE_PITCH + 16 * (i & 63); },
                                   [&](int i, float4 s) {
                                     const int n = nb * 256 + 4 * (i & 63);
                                     put4(static_cast<T*>(p.C) + (row0 + (i >> 6)) * p.ldc + n, s, d, p.N - n);
                                   });
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while its tile is being read
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------------
// Few rows, or few tiles: clusters that split K
// ---------------------------------------------------------------------------------------
// One tile per cluster: 128 rows of B (the MMA's M) by BN rows of A (its N), so that a single token costs an
// MMA of 16 columns and the whole CTA's intake is B. The CTAs of a cluster take consecutive ranges of K; each
// writes its fp32 tile to its own shared memory, and each then sums a share of the columns over all of them, in
// rank order (the same bits every time), and stores it. No workspace, no atomics.
// 1 x 14336 x 4096 NVFP4 in 6.5 us (33 MB of weights: 5.1 TB/s), 23 x 6144 x 1536 MXFP4 in 4.0 (latency: launch, first
// load, the sum over the cluster).
template <int FMT, int BN>
struct Split {
  static constexpr int KA = kAtoms<FMT>;
  static_assert(BN <= 128, "one scale block of A");
  static constexpr int X_BYTES = BN * 128;
  static constexpr int OP_BYTES = kOpBytes + X_BYTES;
  static constexpr int SF_BYTES = 512 * KA * 2;
  static constexpr int TX_BYTES = OP_BYTES + SF_BYTES;
  // up to 64 rows of A two CTAs share an SM (their loads overlap each other's start and end)
  static constexpr int PER_SM = BN <= 64 ? 2 : 1;
  static constexpr int FIT = 220 * 1024 / PER_SM / TX_BYTES;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int THREADS = 192;
  static constexpr int ACC_COLS = BN;
  static constexpr int SFA = ACC_COLS, SFB = SFA + 4 * KA, COLS = SFB + 4 * KA;
  static constexpr int TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;
  static constexpr int OFF_SF = STAGES * OP_BYTES;
  static constexpr int OFF_BAR = OFF_SF + STAGES * SF_BYTES;
  static constexpr int NBAR = 2 * STAGES + 1;
  static constexpr int OFF_SLOT = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM = OFF_SLOT + 16 + 1024;
  static_assert(OFF_SF >= BN * 512, "the fp32 tile fits where the operands were");
  static_assert(OP_BYTES % 1024 == 0 && SMEM <= 232448 && STAGES >= 2, "shared memory");
};

struct SplitParams {
  int M, N, stages_k, splits;
  int64_t ldc;
  void* C;
  const float* da;
  const float* db;
  WaitCtl w;
};

template <int FMT, int BN, typename T>
__global__ void __launch_bounds__(192)
    mm4_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSW,
                     const __grid_constant__ CUtensorMap tmSX, const __grid_constant__ SplitParams p) {
  using C = Split<FMT, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar_full = base + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES, bar_done = bar_empty + 8 * C::STAGES;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  const int splits = p.splits, rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int nb = blockIdx.x / splits, mb = blockIdx.y;  // 128 rows of B, BN rows of A
  const int k0 = static_cast<int>(static_cast<int64_t>(p.stages_k) * rank / splits), k1 = static_cast<int>(static_cast<int64_t>(p.stages_k) * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmSW);
    tma_prefetch_desc(&tmSX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  pdl_wait();
  pdl_trigger();

  bool good = true;  // (epilogue warps)
  if (warp == 0) {
    int issued = 0;
    for (int k = k0; k < k1; ++k, ++issued) {
      const int stage = issued % C::STAGES;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_empty + 8 * stage, ((issued / C::STAGES) & 1) ^ 1u, p.w, DEV_ERR_WAIT_PRODUCER))) break;
      if (elect_one()) {
        const uint32_t sa = base + stage * C::OP_BYTES, sf = base + C::OFF_SF + stage * C::SF_BYTES, fb = bar_full + 8 * stage;
        mbar_arrive_expect_tx(fb, C::TX_BYTES);
        tma_load_2d(sa, &tmW, fb, k * 128, nb * 128);
        tma_load_2d(sa + kOpBytes, &tmX, fb, k * 128, mb * BN);
        tma_load_3d(sf, &tmSW, fb, 0, k * C::KA, nb);
        tma_load_3d(sf + 512 * C::KA, &tmSX, fb, 0, k * C::KA, mb * BN / 128);
      }
      __syncwarp();
    }
    // every load that was issued lands before the CTA can exit, also after a wait that ran out
    for (int s = issued > C::STAGES ? issued - C::STAGES : 0; s < issued; ++s)
      wait_drain(bar_full + 8 * (s % C::STAGES), (s / C::STAGES) & 1, 1000000000ull);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f4(FMT, 128, BN);
    for (int k = k0; k < k1; ++k) {
      const int n = k - k0, stage = n % C::STAGES;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * stage, (n / C::STAGES) & 1, p.w, DEV_ERR_WAIT_MMA))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sa = base + stage * C::OP_BYTES, sf = base + C::OFF_SF + stage * C::SF_BYTES;
        stage_mma<FMT, false, 1>(tmem, sa, sa + kOpBytes, sf, sf + 512 * C::KA, tmem + C::SFA, tmem + C::SFB, idesc, k == k0);
        mma_commit(bar_empty + 8 * stage);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(bar_done);
    __syncwarp();
    if (!wait_drain(bar_done, 0, 4000000000ull)) atomicOr(p.w.err, DEV_ERR_WAIT_TEARDOWN);
  } else {
    good = mbar_wait(bar_done, 0, p.w, DEV_ERR_WAIT_EPILOGUE);
    __syncwarp();
    tc_fence_after();
  }
  const float d = __fmul_rn(p.da != nullptr ? __ldg(p.da) : 1.0f, p.db != nullptr ? __ldg(p.db) : 1.0f);
  T* out = static_cast<T*>(p.C);
  const int live = min(BN, p.M - mb * BN);  // rows of A in this tile
  if (splits == 1) {
    if (warp >= 2 && good) {
      const int q = warp & 3, n = nb * 128 + q * 32 + lane;
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < live; c += 16) {
        uint32_t r[16];
        tmem_ld16(acc + c, r);
        tmem_ld_wait();
        reg_fence(r);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < live && n < p.N) put(out + (mb * BN + c + j) * p.ldc + n, __fmul_rn(__uint_as_float(r[j]), d));
      }
    }
  } else {
    // every load has landed and every MMA is done: the operand ring becomes the fp32 tile [BN][128]
    float* tile = reinterpret_cast<float*>(smem);
    if (warp >= 2 && good) {
      const int q = warp & 3;
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < live; c += 16) {
        uint32_t r[16];
        tmem_ld16(acc + c, r);
        tmem_ld_wait();
        reg_fence(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) tile[(c + j) * 128 + q * 32 + lane] = __uint_as_float(r[j]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    const int c0 = live * rank / splits, c1 = live * (rank + 1) / splits;
    cluster_sum<kMm4Splits, 2>(c0 * 32 + static_cast<int>(threadIdx.x), c1 * 32, C::THREADS, 0, 1, splits, rank, [&](int i) { return base + 16 * i; },
                      [&](int i, float4 s) {
                        const int n = nb * 128 + 4 * (i & 31);
                        put4(out + (mb * BN + (i >> 5)) * p.ldc + n, s, d, p.N - n);
                      });
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while its tile is being read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------------------
// An operand's codes as rows of bytes in boxes of `rows` x 128 bytes, and its scale atoms as
// [128-row block][atom along K][512 bytes] in boxes of `blocks` x the stage's atoms.
bool codes_map(CUtensorMap* m, const void* q, int64_t mn, int64_t k, int rows) {
  const uint64_t pitch = static_cast<uint64_t>(fp4::row_bytes(k));
  return encode_tmap_2d(m, q, CU_TENSOR_MAP_DATA_TYPE_UINT8, pitch, static_cast<uint64_t>(mn), pitch, 128, static_cast<uint32_t>(rows), 128);
}
bool scales_map(CUtensorMap* m, const void* sf, int fmt, int64_t mn, int64_t k, int blocks) {
  const uint64_t atoms = static_cast<uint64_t>(fp4::atoms_along(fmt, k));
  return encode_tmap_3d(m, sf, CU_TENSOR_MAP_DATA_TYPE_UINT32, 128, atoms, static_cast<uint64_t>((mn + 127) / 128), 512, atoms * 512, 128,
                        fmt == 0 ? 4 : 2, static_cast<uint32_t>(blocks));
}

// Once per device and kernel: the shared-memory limit; and per cluster size (up to 8), how many clusters are resident
// at once (0: none fits, which is no error here).
template <auto Kernel>
cudaError_t prepare(int smem, int threads, int cluster, int* resident) {
  static bool done[64] = {}, asked[64][9] = {};
  static int count[64][9] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  if (!asked[dev][cluster]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(Kernel), &cfg);
    if (e == cudaErrorInvalidClusterSize) {
      cudaGetLastError();
      n = 0;
    } else if (e != cudaSuccess) {
      return e;
    }
    count[dev][cluster] = n;
    asked[dev][cluster] = true;
  }
  *resident = count[dev][cluster];
  return cudaSuccess;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <int FMT, bool F32, bool SPLIT>
cudaError_t launch_pair(const Mm4Args& g, int splits, cudaStream_t stream, const char** why) {
  using C = Pair<FMT>;
  int clusters = 0;
  const cudaError_t e = prepare<mm4_pair_kernel<FMT, F32, SPLIT>>(C::SMEM, C::THREADS, 2 * splits, &clusters);
  if (e != cudaSuccess) return e;
  if (clusters <= 0) return cudaErrorInvalidConfiguration;
  CUtensorMap a, b, sa, sb, c;
  if (!codes_map(&a, g.A, g.M, g.K, 128) || !codes_map(&b, g.B, g.N, g.K, 128) || !scales_map(&sa, g.sfa, FMT, g.M, g.K, 1) ||
      !scales_map(&sb, g.sfb, FMT, g.N, g.K, 2) ||
      !encode_tmap_2d(&c, g.C, F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.N, g.M, g.ldc * (F32 ? 4 : 2),
                      F32 ? 32 : 64, 32, 128)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  PairParams p{};
  p.M = static_cast<int>(g.M);
  p.N = static_cast<int>(g.N);
  p.num_m = static_cast<int>((g.M + 255) / 256);
  p.num_n = static_cast<int>((g.N + 255) / 256);
  p.tiles = p.num_m * p.num_n;
  p.stages_k = static_cast<int>((g.K + kStageK - 1) / kStageK);
  p.group_m = 16;
  p.splits = splits;
  p.C = g.C;
  p.ldc = g.ldc;
  p.da = g.da;
  p.db = g.db;
  p.w = wait_ctl();
  if constexpr (SPLIT) {
    return launch_cluster(mm4_pair_kernel<FMT, F32, true>, dim3(2 * splits * p.tiles), C::THREADS, C::SMEM, 2 * splits, stream, a, b, sa, sb, c, p);
  } else {
    const int slots = p.tiles < clusters ? p.tiles : clusters;
    return launch_cluster(mm4_pair_kernel<FMT, F32, false>, dim3(2 * slots), C::THREADS, C::SMEM, 2, stream, a, b, sa, sb, c, p);
  }
}

template <int FMT, int BN, typename T>
cudaError_t launch_split(const Mm4Args& g, int splits, cudaStream_t stream, const char** why) {
  using C = Split<FMT, BN>;
  for (int n = 0;; --splits) {  // clusters that the device holds
    const cudaError_t e = prepare<mm4_split_kernel<FMT, BN, T>>(C::SMEM, C::THREADS, splits, &n);
    if (e != cudaSuccess) return e;
    if (n > 0) break;
    if (splits == 1) return cudaErrorInvalidConfiguration;
  }
  CUtensorMap w, x, sw, sx;
  if (!codes_map(&w, g.B, g.N, g.K, 128) || !codes_map(&x, g.A, g.M, g.K, BN) || !scales_map(&sw, g.sfb, FMT, g.N, g.K, 1) ||
      !scales_map(&sx, g.sfa, FMT, g.M, g.K, 1)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  SplitParams p{};
  p.M = static_cast<int>(g.M);
  p.N = static_cast<int>(g.N);
  p.stages_k = static_cast<int>((g.K + kStageK - 1) / kStageK);
  p.splits = splits;
  p.ldc = g.ldc;
  p.C = g.C;
  p.da = g.da;
  p.db = g.db;
  p.w = wait_ctl();
  const dim3 grid(static_cast<unsigned>((g.N + 127) / 128 * splits), static_cast<unsigned>((g.M + BN - 1) / BN));
  return launch_cluster(mm4_split_kernel<FMT, BN, T>, grid, C::THREADS, C::SMEM, splits, stream, w, x, sw, sx, p);
}

// How many clusters of each number of splits the current device holds at once, asked once.
template <int FMT, typename T>
cudaError_t clusters_held(const Mm4Clusters** out) {
  static Mm4Clusters all[64];
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[dev]) {
    using P = Pair<FMT>;
    using S = Split<FMT, 128>;
    for (int s = 1; s <= kMm4PairSplits && e == cudaSuccess; ++s)
      e = s == 1 ? prepare<mm4_pair_kernel<FMT, sizeof(T) == 4, false>>(P::SMEM, P::THREADS, 2, &all[dev].pair[s])
                 : prepare<mm4_pair_kernel<FMT, sizeof(T) == 4, true>>(P::SMEM, P::THREADS, 2 * s, &all[dev].pair[s]);
    for (int s = 1; s <= kMm4Splits && e == cudaSuccess; ++s) e = prepare<mm4_split_kernel<FMT, 128, T>>(S::SMEM, S::THREADS, s, &all[dev].one[s]);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  *out = &all[dev];
  return cudaSuccess;
}

template <int FMT, typename T>
cudaError_t launch_as(const Mm4Args& g, cudaStream_t stream, const char** why) {
  Mm4Plan p{0, 0};
  if (g.M <= 64) {
    p = mm4_plan_few_rows(g.M, g.N, g.K, num_sms());
  } else {
    const Mm4Clusters* fit = nullptr;
    const cudaError_t e = clusters_held<FMT, T>(&fit);
    if (e != cudaSuccess) return e;
    p = mm4_plan(g.M, g.N, g.K, num_sms(), *fit);
    if (p.splits == 0) {
      *why = "the device holds no cluster of two CTAs";
      return cudaErrorInvalidConfiguration;
    }
  }
  switch (p.bn) {
    case 0:
      return p.splits > 1 ? launch_pair<FMT, sizeof(T) == 4, true>(g, p.splits, stream, why) : launch_pair<FMT, sizeof(T) == 4, false>(g, 1, stream, why);
    case 16: return launch_split<FMT, 16, T>(g, p.splits, stream, why);
    case 32: return launch_split<FMT, 32, T>(g, p.splits, stream, why);
    case 64: return launch_split<FMT, 64, T>(g, p.splits, stream, why);
    default: return launch_split<FMT, 128, T>(g, p.splits, stream, why);
  }
}

}  // namespace

cudaError_t launch_mm4(const Mm4Args& g, cudaStream_t stream, const char** why) {
  if (wait_ctl().err == nullptr) {
    *why = "device error word unavailable";
    return cudaErrorInvalidDevice;
  }
  if (g.f32) return g.fmt == 0 ? launch_as<0, float>(g, stream, why) : launch_as<1, float>(g, stream, why);
  return g.fmt == 0 ? launch_as<0, __nv_bfloat16>(g, stream, why) : launch_as<1, __nv_bfloat16>(g, stream, why);
}

}  // namespace fp8gb
