// paged_attention.cu -- attention of new tokens over a paged cache on the tensor cores.
//
//   out_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = exp(scale q_i . k_j - m_i)
//
// in one pass over the keys with a running reference m: per tile of 128 keys S = Q K^T (tcgen05, bf16, fp32 in tensor memory), the
// weights in registers, P = bf16(weights) back to tensor memory over S, O += P V with P read from there. A CTA stays on its
// SM and works through a run of tiles (attend_walk.cuh); its warps divide the work:
//   0-3 (and 4-7)  weights, one thread per row: 128 rows of a tile each
//   the next 4 or 8  keys and values on their way: 8-bit codes into bf16 (a code times a power of two: exact down to bf16's smallest numbers), and what must not be
//                  multiplied by a weight of zero out of the last tiles (below)
//   the last ones  copies (TMA, one box per page), tensor-core instructions (a thread per tile of rows)
// Three forms (chosen at the end of this file): two tiles of rows over the same keys, one's weights worked out while the other is on the tensor cores (NQ 2);
// one tile (NQ 1, bf16 only); and SPREAD, 32 rows four times in a tile, whose copies weigh a quarter of a tile's keys each (the other
// keys' weights stay zero) and are added up at the unit's end, so that a single token's few rows still have four warps.
//
// The reference moves only where a row's maximum passes it by more than 8 (in log2 of the weights; below, exp cannot overflow
// and fp32 sums lose nothing): then O in tensor memory and the sum are scaled, otherwise O is never touched.
//
// P is rounded to bf16 because the tensor cores take both operands of the second product in 16 bits; the sum of the weights is of the unrounded ones, so
// that the roundings (half a step, 2^-9 on average) stay independent errors of the terms and not of the whole.
//
// Measured (4 query heads to each of 8 cache heads, D 128): 64 tokens over 4096 keys each 172 us, 6.2 TB/s, 0.92 of a copy's rate: memory; the
// same in 8 bits 147 us, 3.8 TB/s: shared memory's bandwidth (copies, conversion and tensor cores together use 0.85 of it). A chunk
// of 2048 tokens over 16384 keys 364 us by itself, 382 in a loop under the power limit, 1416 and 1350 TFLOP/s, 0.74 and 0.71 of a large product's
// rate: the weights' arithmetic, of which a tile's 64 keys take some 1700 clocks and their products 1370. One token over 100 keys 8 us
// (D 64: 7): the chain launch, lengths, page table, keys, scores, weights, output.
//
// Masked places. Weights are set, not added to, so keys may be anything. A value that is not finite would make 0 * inf of a
// weight of zero: in tiles with keys that some row does not see (the last ones, and the first ones of a window) values
// behind the end become zero, and others that are not finite become zero as well and are added at the end to the rows that see them.
//
// A unit cut by the end of a CTA's run leaves sum, reference and O of each part in the workspace; the CTA that finds itself the last
// of them (a counter) adds them up in the order of the parts, so the result does not depend on who that is.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>
#include <numeric>

#include "attend_walk.cuh"
#include "heads.cuh"
#include "kernels.h"

namespace fp8gb {
namespace {

using namespace attend;
using heads::bf16;

constexpr int kPanel = 16384;        // 128 rows of 128 bytes
constexpr int kCounterBytes = 4096;  // of the workspace: two counters per CTA
constexpr int kMaxCtas = 160;        // (152 SMs; what a join holds of each part has to fit into shared memory)
constexpr int kJoinBytes = 200 * 1024;  // of shared memory
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
template <int D, bool MX, int NQ, bool SPREAD>
struct Form {
  static constexpr int PANELS = D / 64;
  static constexpr int TILE = PANELS * kPanel;  // 128 rows of bf16
  // keys and values: groups of 8 rows, each panel's 8 x 128 bytes after the other (queries: a panel's 128 rows together)
  static constexpr int GROUP = PANELS * 1024;
  // Stages of keys and values: in turn, or (8-bit, one tile of rows: two groups of warps convert them side by side) each their own. Values
  // wait for their weights and are held three times as long as keys.
  static constexpr bool APART = MX && NQ == 1;
  static constexpr int KEYS = D == 128 ? 1 : 2, STAGES = MX ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int QBUFS = APART && D == 128 ? 1 : 2;  // buffers of queries (NQ 2: one for each tile)
  static __device__ __forceinline__ int stage_of(int n, int kv) { return !APART ? (2 * n + kv) % STAGES : kv == 0 ? n % KEYS : KEYS + n % (STAGES - KEYS); }
  static __device__ __forceinline__ uint32_t phase_of(int n, int kv) { return (!APART ? (2 * n + kv) / STAGES : kv == 0 ? n / KEYS : n / (STAGES - KEYS)) & 1; }
  static constexpr int RAW = 128 * D, UNITS = 4 * D;  // 128 rows of codes (rows of 128: their 16-byte pieces in the copy's swizzle), and their units
  static constexpr int RAWS = MX ? (D == 128 ? (NQ == 1 ? 4 : 3) : (NQ == 1 ? 8 : 6)) : 0;
  // warps: weights, then those that work on keys and values on their way, one for the copies, one or two for the tensor cores
  static constexpr int PREP_WARP = NQ == 1 ? 4 : 8, PREP_WARPS = 12 - PREP_WARP;
  // On one 8-bit tile; one tile of rows: keys and values side by side (64 tokens over 4096 keys of 8 heads of 128: 144 us; with one stage for
  // each 156, and 165 while the lanes that read a row's codes and write its panels met in the banks; 8 warps on each tile, three stages in turn,
  // 174 beside 170 then). Shared memory is what they wait for: the codes in and out, the bf16 in, and each read once by the tensor cores.
  static constexpr int GROUP_WARPS = 4;
  // Copies: one tile of rows: a warp for the keys and one for the values (8-bit: one warp for both took 2180 clocks an item, of which
  // the conversion took 790). Two: keys and values share stages, so one.
  static constexpr int COPY_WARPS = NQ == 1 ? 2 : 1;
  static constexpr int COPY_WARP = PREP_WARP + PREP_WARPS, MMA_WARP = COPY_WARP + COPY_WARPS, WARPS = MMA_WARP + NQ, THREADS = 32 * WARPS;
  static_assert(NQ == 2 || NQ == 1, "tiles");
  static_assert(NQ == 1 || !SPREAD, "one tile of spread rows");
  static constexpr int OFF_KV = QBUFS * TILE;
  static constexpr int OFF_RAW = OFF_KV + STAGES * TILE;
  static constexpr int OFF_UNITS = OFF_RAW + RAWS * RAW;
  // where the four copies of spread rows are added up: in their queries' buffer, or beside it where the next unit's come into it
  static constexpr int OFF_SHARE = OFF_UNITS + RAWS * UNITS, SHARE = SPREAD && QBUFS == 1 ? 16384 : 0, OFF_END = OFF_SHARE + SHARE;
  static constexpr int OFF_BAR = OFF_END > kJoinBytes ? OFF_END : kJoinBytes;
  static constexpr int NBAR = 4 + 3 * STAGES + 2 * RAWS + 12 + 2;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_STATS = OFF_MISC + 512;  // (reference, sum) of each row, SPREAD: of each warp's rows
  static constexpr int SMEM = OFF_STATS + 1024 * NQ + 1024;
  // A wait names a phase by its parity, so whoever waits on a barrier has to see all of its phases. Where keys and values have
  // different waiters (the warps that look at bf16 values, the two groups that convert 8-bit tiles) a stage is always
  // one or the other's.
  static_assert(APART ? RAWS % 2 == 0 : MX || STAGES % 2 == 0, "stages");
  static_assert(RAW % 1024 == 0 && OFF_RAW % 1024 == 0 && OFF_BAR % 8 == 0 && SMEM <= 232448, "shared memory");
  static_assert(OFF_RAW >= 4 * kAttendMaxSeqs, "room for the sequences' costs");
};

struct Params {
  Attention a;
  Cache c;
  Batch b;
  int group, tokens_per_tile, capacity;
  int group_inverse;  // ceil(2^16 / group): (r * group_inverse) >> 16 is r / group for r < 128
  float c2;   // |scale| log2 e
  bool flip;  // scale < 0
  int page_steps, head_steps;  // of a bf16 cache's pages and heads in its tensor maps' last dimension
  char* parts;
  unsigned* counters;
  WaitCtl w;
};

// A cut tile of rows whose parts are all there: rows `rows` from token `token` and head `head` on, of CTAs c0 .. c1.
struct Join {
  int64_t token;
  int head, rows, c0, c1;
};

// What is not in rings, at OFF_MISC.
struct Misc {
  Place start;
  int64_t total;
  int runs;
  uint32_t tmem;
  Join join[4];     // what this CTA adds up at its end: of each tile of rows, the run's first unit and its last
  uint32_t bad[8];  // of each raw tile, the boxes whose page is outside the cache
  int dirty[16];  // the last segment with tiles, of those with this number modulo 16, that holds values that are not finite in edge tiles
};
static_assert(sizeof(Misc) <= 512 && 8 * kMaxCtas <= kCounterBytes, "misc");
static_assert(kJoinBytes >= kMaxCtas * (256 + 2 * 512), "eight columns of a block of all parts");

struct Sequences {
  const Batch& b;
  int capacity, seqs;
  __device__ __forceinline__ Seq seq(int s) const {
    return seq_of(__ldg(b.q_start + s), __ldg(b.q_start + s + 1), __ldg(b.kv_len + s), static_cast<int>(b.tokens), capacity);
  }
};

// ---- where this CTA's run begins -------------------------------------------------------------------------------------
// Few sequences of few blocks: a lane for each, every warp for itself (one token over 1000: 2 us of 12 with
// the general way below).
__device__ bool find_start_of_few(const Params& p, const Sequences& src, int per, Misc* misc) {
  const int lane = threadIdx.x & 31;
  if (src.seqs > 32) return false;
  Seq q{0, 0, 0, 0};
  if (lane < src.seqs) q = src.seq(lane);
  if (__syncthreads_or(q.n > 4 * per)) return false;  // (all of the CTA alike, whatever a length does meanwhile)
  int mine = 0;
  for (int b = 0; b * per < q.n; ++b) mine += items_of(q, b, per, p.a.window);
  const int64_t all = static_cast<int64_t>(mine) * p.c.heads;
  int64_t upto = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += x;
  }
  const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  const int runs = static_cast<int>(min(total, static_cast<int64_t>(gridDim.x)));  // none of them empty
  const bool works = static_cast<int>(blockIdx.x) < runs;
  const int64_t begin = works ? begin_of(total, blockIdx.x, runs) : 0, end = works ? begin_of(total, blockIdx.x + 1, runs) : 0;
  if (threadIdx.x == 0) {
    misc->total = total;
    misc->runs = runs;
    misc->start.item = begin;
    misc->start.end = end;
  }
  if (threadIdx.x < 32 && works && upto - all <= begin && begin < upto) {
    const int64_t at = begin - (upto - all);
    const int head = static_cast<int>(quotient(at, mine));
    int off = static_cast<int>(at - static_cast<int64_t>(head) * mine), block = 0;
    for (int n; off >= (n = items_of(q, block, per, p.a.window)); ++block) off -= n;
    misc->start.seq = lane;
    misc->start.head = head;
    misc->start.block = block;
    misc->start.off = off;
  }
  return true;
}

template <int kThreads>
__device__ void find_start(const Params& p, const Sequences& src, int per, uint32_t* cost, Misc* misc, int64_t* share) {
  constexpr uint32_t kLong = 0xFFFFFFFFu;
  if (find_start_of_few(p, src, per, misc)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, seqs = src.seqs;
  bool some_long = false;
  for (int s = tid; s < seqs; s += kThreads) {
    const Seq q = src.seq(s);
    uint32_t n = 0;
    if (q.n > 4 * per) {
      n = kLong;
      some_long = true;
    } else {
      for (int b = 0; b * per < q.n; ++b) n += items_of(q, b, per, p.a.window);
    }
    cost[s] = n;
  }
  if (__syncthreads_or(some_long)) {
    for (int s = warp; s < seqs; s += kThreads / 32) {
      if (cost[s] != kLong) continue;
      const Seq q = src.seq(s);
      uint32_t n = 0;
      for (int b = lane; static_cast<int64_t>(b) * per < q.n; b += 32) n += items_of(q, b, per, p.a.window);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
      __syncwarp();
      if (lane == 0) cost[s] = n;
    }
    __syncthreads();
  }
  const int chunk = (seqs + kThreads - 1) / kThreads, s0 = min(tid * chunk, seqs), s1 = min(s0 + chunk, seqs);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += static_cast<int64_t>(cost[s]) * p.c.heads;
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) share[warp] = upto;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += share[w];
    total += share[w];
  }
  const int runs = static_cast<int>(min(total, static_cast<int64_t>(gridDim.x)));  // none of them empty
  const bool works = static_cast<int>(blockIdx.x) < runs;
  const int64_t begin = works ? begin_of(total, blockIdx.x, runs) : 0, end = works ? begin_of(total, blockIdx.x + 1, runs) : 0;
  if (tid == 0) {
    misc->total = total;
    misc->runs = runs;
    misc->start.item = begin;
    misc->start.end = end;
  }
  int64_t at = before + upto - mine;
  if (begin < end && at <= begin && begin < at + mine) {
    int s = s0;
    for (; s < s1 - 1 && at + static_cast<int64_t>(cost[s]) * p.c.heads <= begin; ++s) at += static_cast<int64_t>(cost[s]) * p.c.heads;
    misc->start.seq = s;
    misc->start.head = static_cast<int>((begin - at) / cost[s]);
    misc->start.off = static_cast<int>((begin - at) % cost[s]);
  }
  __syncthreads();
  if (warp == 0 && begin < end) {
    const Seq q = src.seq(misc->start.seq);
    uint32_t rest = static_cast<uint32_t>(misc->start.off);
    int block = 0;
    for (int b0 = 0; static_cast<int64_t>(b0) * per < q.n; b0 += 32) {
      const int64_t b = b0 + lane;
      const uint32_t n = b * per < q.n ? items_of(q, static_cast<int>(b), per, p.a.window) : 0u;
      uint32_t upto_b = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto_b, o);
        if (lane >= o) upto_b += x;
      }
      const uint32_t all = __shfl_sync(0xFFFFFFFFu, upto_b, 31);
      if (rest < all) {
        const int l = __ffs(__ballot_sync(0xFFFFFFFFu, upto_b > rest)) - 1;
        rest -= __shfl_sync(0xFFFFFFFFu, upto_b - n, l);
        block = b0 + l;
        break;
      }
      rest -= all;
    }
    __syncwarp();
    if (lane == 0) {
      misc->start.block = block;
      misc->start.off = static_cast<int>(rest);
    }
  }
}

// ---- small pieces ----------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint64_t both(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Whether either half of a word is a bf16 that is not finite.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  const uint32_t bad = not_finite(w);
  return w & ~((bad & 0x8000u ? 0xFFFFu : 0u) | (bad & 0x80000000u ? 0xFFFF0000u : 0u));
}

// 16 E4M3 codes as bf16, times f. A code's exponent and mantissa in bf16's places are the value times 2^-120 (subnormals
// included), exactly: each half takes a code and its sign's eight copies, moved up by four.
__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t w) {
  __nv_bfloat162 v;
  memcpy(&v, &w, 4);
  return v;
}
__device__ __forceinline__ uint32_t times(uint32_t w, __nv_bfloat162 f) {
  const __nv_bfloat162 v = __hmul2(as_pair(w), f);
  uint32_t r;
  memcpy(&r, &v, 4);
  return r;
}
__device__ __forceinline__ void decode16(const uint4& x, __nv_bfloat162 f, uint32_t (&y)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t a, b;
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w[e]));
    asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(b) : "r"(w[e]));
    y[2 * e] = times((a << 4) & 0x87F087F0u, f);
    y[2 * e + 1] = times((b << 4) & 0x87F087F0u, f);
  }
}
__device__ __forceinline__ __nv_bfloat162 bf16_pair(uint32_t bits) {
  const uint32_t w = bits | (bits << 16);
  __nv_bfloat162 v;
  memcpy(&v, &w, 4);
  return v;
}

// What a row's elements are divided by: 0 for a row that saw nothing, NaN under a score of +infinity (infinity over infinity).
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.0f ? 0.0f : isinf(sum) ? __int_as_float(0x7FFFFFFF) : 1.0f / sum; }

// A value of the cache that is not finite, or 0.
template <bool MX, int D>
__device__ float unusual(const Params& p, int64_t row, int64_t unit, int d) {
  float v;
  if constexpr (MX) {
    const uint32_t u = p.c.v_scale[unit + d / 32], b = static_cast<const uint8_t*>(p.c.v)[row + d];
    if (u == 0xFFu) return __int_as_float(0x7FFFFFFF);
    v = __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7Fu) << 20)) * 0x1p120f * (u == 0u ? 0x1p-127f : __uint_as_float(u << 23));
  } else {
    v = __bfloat162float(static_cast<const bf16*>(p.c.v)[row + d]);
  }
  return isfinite(v) ? 0.0f : v;
}

// After a wait that ran out: time for the copies in flight to land (microseconds) before the CTA can exit.
__device__ __noinline__ void settle() {
  const unsigned long long t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 200000ull) {
  }
}

// ---- a tile's rows, and its parts ------------------------------------------------------------------------------------
// Row r of a tile that begins at a token and query head.
__device__ __forceinline__ bf16* row_of(const Params& p, int64_t token, int head, int r) {
  const int tk = (r * p.group_inverse) >> 16, hd = r - tk * p.group;
  return static_cast<bf16*>(p.a.out) + (token + tk) * p.a.ld_out + (static_cast<int64_t>(head) + hd) * p.a.hs_out;
}
__device__ __forceinline__ void put_lse(const Params& p, int64_t token, int head, int r, float reference, float sum) {
  if (p.a.lse == nullptr) return;
  const int tk = (r * p.group_inverse) >> 16, hd = r - tk * p.group;
  p.a.lse[(token + tk) * p.a.q_heads + head + hd] = sum == 0.0f ? -INFINITY : (reference + log2f(sum)) * kLn2;
}
// The part of a cut unit (its first CTA c0) that a CTA leaves in the workspace: (reference, sum) of each row, then O by
// blocks of 32 rows, in a block four columns of all its rows after the other (a warp, a thread per row, writes without gaps).
template <int D, int NQ>
__device__ __forceinline__ char* part_at(const Params& p, int c0, int cta, int q) {
  return p.parts + (static_cast<int64_t>(2 * cta + (cta == c0 ? 1 : 0)) * NQ + q) * (128 * (D + 2) * 4);
}

// A unit's parts added up, in their order, by the whole CTA at its end, when shared memory is free: for as many blocks of 32 rows of all
// parts as fit (or some columns of one) their references and sums become weights, then the rows' elements are added. What bounds it is the
// way to L2 and back, and code that comes once and from far: short loops over bulk copies.
template <int D, int NQ, int kThreads>
__device__ __noinline__ bool join_parts(const Params& p, const Join u, int q, uint8_t* smem, float* inverse, uint32_t bar, uint32_t& phase) {
  constexpr int kAll = D / 4, kLanes = 8;  // columns by fours; threads for a row's statistics
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, parts = u.c1 - u.c0 + 1;
  const int whole = kJoinBytes / (parts * (256 + kAll * 512)), step = 32 * most(whole, 1);
  const int wide = whole > 0 ? kAll : (kJoinBytes / parts - 256) / 512 & ~1;  // columns by fours at once, an even number
  __threadfence();
  if (u.rows * kAll <= kThreads && parts <= 32) {  // few rows: a thread for four elements, its reference and sum on the way
    if (tid >= u.rows * kAll) return true;
    static_assert(kThreads / kAll <= 32, "rows of one block, as they lie in the parts");
    const int d = tid / u.rows, r = tid - d * u.rows;
    float top = -INFINITY, sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int c = 0; c < parts; c += 8) {
      float2 x[8];
      float4 y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const char* at = part_at<D, NQ>(p, u.c0, u.c0 + least(c + b, parts - 1), q);
        x[b] = __ldcg(reinterpret_cast<const float2*>(at) + r);
        y[b] = __ldcg(reinterpret_cast<const float4*>(at + 1024) + tid);
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (c + b >= parts || x[b].y == 0.0f) continue;  // 0: a part that saw nothing
        const float to = fmaxf(top, x[b].x), f = exp2_of(top - to), w = exp2_of(x[b].x - to);
        top = to;
        sum = fmaf(w, x[b].y, sum * f);
        o.x = fmaf(w, y[b].x, o.x * f), o.y = fmaf(w, y[b].y, o.y * f), o.z = fmaf(w, y[b].z, o.z * f), o.w = fmaf(w, y[b].w, o.w * f);
      }
    }
    if (d == 0) put_lse(p, u.token, u.head, r, top, sum);
    const float inv = inverse_of(sum);
    *reinterpret_cast<uint2*>(row_of(p, u.token, u.head, r) + 4 * d) =
        inv == 0.0f ? make_uint2(0u, 0u) : make_uint2(heads::pack(o.x * inv, o.y * inv), heads::pack(o.z * inv, o.w * inv));
    return true;
  }
  const uint32_t base = smem_u32(smem);
  const float2* ml = reinterpret_cast<const float2*>(smem);  // [parts][rows of this step, up to 32 more of them]
#pragma unroll 1
  for (int r0 = 0; r0 < u.rows; r0 += step) {
    const int rows = least(step, u.rows - r0), ml_rows = (rows + 1) & ~1;
#pragma unroll 1
    for (int d0 = 0; d0 < kAll; d0 += wide) {
      const int columns = least(wide, kAll - d0), o_bytes = rows * columns * 16, o_at = parts * ml_rows * 8;
      fence_proxy_async();
      __syncthreads();
      if (warp == 0) {
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(parts * (o_bytes + ml_rows * 8)));
        __syncwarp();
#pragma unroll 1
        for (int c = lane; c < parts; c += 32) {
          const char* at = part_at<D, NQ>(p, u.c0, u.c0 + c, q);
          bulk_load(base + c * ml_rows * 8, at + 8 * r0, ml_rows * 8, bar);
          bulk_load(base + o_at + c * o_bytes, at + 1024 + (r0 * kAll + d0 * rows) * 16, o_bytes, bar);
        }
      }
      const bool ok = mbar_wait(bar, phase, p.w, DEV_ERR_WAIT_EPILOGUE);
      if (!__syncthreads_and(ok)) return false;
      phase ^= 1u;
      float2* weight = const_cast<float2*>(ml);
#pragma unroll 1
      for (int r1 = 0; r1 < rows; r1 += kThreads / kLanes) {
        const int r = r1 + tid / kLanes, l = tid % kLanes;
        float top = -INFINITY, sum = 0.0f;
        if (r < rows) {
#pragma unroll 2
          for (int c = l; c < parts; c += kLanes) top = fmaxf(top, ml[c * ml_rows + r].x);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (top == -INFINITY) top = 0.0f;
        if (r < rows) {
#pragma unroll 2
          for (int c = l; c < parts; c += kLanes) {
            const float2 x = ml[c * ml_rows + r];
            const float w = exp2_of(x.x - top);
            weight[c * ml_rows + r].x = w;
            sum = fmaf(w, x.y, sum);
          }
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (r < rows && l == 0) {
          if (d0 == 0) put_lse(p, u.token, u.head, r0 + r, top, sum);
          inverse[r] = inverse_of(sum);
        }
      }
      __syncthreads();
      const int pairs = columns / 2, blocks = (rows + 31) / 32;
#pragma unroll 1
      for (int x = warp; x < blocks * pairs; x += kThreads / 32) {  // 8 columns of a block, a lane per row
        const int block = x / pairs, d = x - block * pairs, across = least(rows - 32 * block, 32), r = lane;
        if (r >= across) continue;
        const float4* from = reinterpret_cast<const float4*>(smem + o_at) + 32 * block * columns + 2 * d * across + r;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), e = o;
#pragma unroll 2
        for (int c = 0; c < parts; ++c) {
          const float2 w = ml[c * ml_rows + 32 * block + r];
          const float4 a = from[c * (o_bytes / 16)], b = from[c * (o_bytes / 16) + across];
          if (w.y == 0.0f) continue;  // a part that saw nothing
          o.x = fmaf(w.x, a.x, o.x), o.y = fmaf(w.x, a.y, o.y), o.z = fmaf(w.x, a.z, o.z), o.w = fmaf(w.x, a.w, o.w);
          e.x = fmaf(w.x, b.x, e.x), e.y = fmaf(w.x, b.y, e.y), e.z = fmaf(w.x, b.z, e.z), e.w = fmaf(w.x, b.w, e.w);
        }
        const float inv = inverse[32 * block + r];
        uint4 packed = make_uint4(heads::pack(o.x * inv, o.y * inv), heads::pack(o.z * inv, o.w * inv), heads::pack(e.x * inv, e.y * inv), heads::pack(e.z * inv, e.w * inv));
        if (inv == 0.0f) packed = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(row_of(p, u.token, u.head, r0 + 32 * block + r) + 4 * d0 + 8 * d) = packed;
      }
    }
  }
  return true;
}

template <int D, bool MX, int NQ, bool SPREAD>
__global__ void __launch_bounds__(Form<D, MX, NQ, SPREAD>::THREADS, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Params p) {
  using F = Form<D, MX, NQ, SPREAD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Misc* misc = reinterpret_cast<Misc*>(smem + F::OFF_MISC);
  const uint32_t q_full = base + F::OFF_BAR, q_empty = q_full + 16, kv_full = q_empty + 16, kv_empty = kv_full + 8 * F::STAGES;
  const uint32_t raw_full = kv_empty + 8 * F::STAGES, raw_empty = raw_full + 8 * F::RAWS, s_full = raw_empty + 8 * F::RAWS;
  const uint32_t p_ready = s_full + 32, o_done = p_ready + 32, v_fixed = o_done + 32, bar_final = v_fixed + 8 * F::STAGES, bar_join = bar_final + 8;
  const int per = NQ * p.tokens_per_tile;
  const Sequences src{p.b, p.capacity, p.b.seqs};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, F::SHARE == 0 && SPREAD ? 2 : NQ);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
    }
    for (int i = 0; i < F::STAGES; ++i) {
      mbar_init(kv_full + 8 * i, MX ? F::GROUP_WARPS : 1);
      mbar_init(kv_empty + 8 * i, NQ);
      mbar_init(v_fixed + 8 * i, F::PREP_WARPS);
    }
    for (int i = 0; i < F::RAWS; ++i) {
      mbar_init(raw_full + 8 * i, 33);  // each lane's copies of units, and the codes'
      mbar_init(raw_empty + 8 * i, F::GROUP_WARPS);
    }
    mbar_init(bar_final, NQ);
    mbar_init(bar_join, 1);
    fence_mbar_init();
    for (int i = 0; i < 16; ++i) misc->dirty[i] = -1;
    for (int i = 0; i < 4; ++i) misc->join[i].rows = 0;
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == F::MMA_WARP) {
    tmem_alloc(smem_u32(&misc->tmem), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  // (the costs lie where the tiles will: written before the barrier, fenced against the copies)
  find_start<F::THREADS>(p, src, per, reinterpret_cast<uint32_t*>(smem), misc, reinterpret_cast<int64_t*>(smem + F::OFF_MISC - 8 * F::NBAR - 256));
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  const int64_t total = misc->total;
  const int runs = misc->runs;
  Walk<Sequences> k(src, misc->start, p.c.heads, per, p.a.window);
  // Scores and weights in tensor memory. SPREAD: two tiles' scores in turn, their weights beside them. Otherwise a tile's scores in two
  // halves of 64 keys (slot 2 q + half), each followed over itself by its weights: one half is on the tensor cores while the
  // other's weights are worked out (with a tile's scores in one piece the tensor cores waited for half of the time).
  auto scores_at = [&](int slot) { return tmem + (SPREAD ? 128 : 64) * slot; };
  auto weights_at = [&](int slot) { return SPREAD ? tmem + 384 + 64 * slot : scores_at(slot) + 32; };

  if (warp >= F::COPY_WARP && warp < F::MMA_WARP) {
    // ---- copies ------------------------------------------------------------------------------------------------------
    const int row_bits = least(p.c.page_bits, 7), rows = 1 << row_bits;  // of a box
    const int kv0 = F::COPY_WARPS == 2 ? warp - F::COPY_WARP : 0, kv1 = F::COPY_WARPS == 2 ? kv0 + 1 : 2;
    bool ok = true;
    int n = 0;  // items so far
    for (; ok && k.live(); k.next()) {
      if (k.a >= k.b) continue;
      // 64 pages of the table ahead, a lane 2 of them: pages[0] from page index `window` on, pages[1] the 32 after
      const int32_t* table = p.b.page_table + k.at.seq * p.b.ld_table;
      const int ends = ((k.s.seen - 1) >> p.c.page_bits) + 1;  // pages of the sequence
      auto page_at = [&](int i) {  // -1 outside the cache
        const int page = i < ends ? __ldg(table + i) : -1;
        return page >= 0 && page < p.c.pages ? page : -1;
      };
      int window = (k.a * kTile) >> p.c.page_bits;
      int pages0 = page_at(window + lane), pages1 = page_at(window + 32 + lane);
      auto load_queries = [&]() {
        const int buf = NQ == 1 ? k.filled % F::QBUFS : 0, use = NQ == 1 ? k.filled / F::QBUFS : k.filled;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(q_empty + 8 * buf, (use & 1) ^ 1u, p.w, DEV_ERR_WAIT_PRODUCER));
        if (!ok) return;
        const int t0 = k.at.block * per, tiles = NQ == 2 && t0 + p.tokens_per_tile < k.s.n ? 2 : 1;
        if (elect_one()) {
          mbar_arrive_expect_tx(q_full + 8 * buf, static_cast<uint32_t>((SPREAD ? 4 : tiles) * p.tokens_per_tile * p.group * D * 2));
          for (int i = 0; i < (SPREAD ? 4 : tiles); ++i)
#pragma unroll
            for (int j = 0; j < F::PANELS; ++j)
              tma_load_3d(base + (NQ == 1 ? buf : i) * F::TILE + j * kPanel + (SPREAD ? i * 4096 : 0), &tm_q, q_full + 8 * buf, 64 * j, k.at.head * p.group,
                          k.s.first + t0 + (SPREAD ? 0 : i * p.tokens_per_tile));
        }
        __syncwarp();
      };
      if (F::QBUFS == 2 && kv0 == 0) load_queries();
      if (!ok) break;
      auto page_of = [&](int i) {  // page i of the sequence, each lane its own i, all within the window
        const int at = i - window, lo = __shfl_sync(0xFFFFFFFFu, pages0, at & 31), hi = __shfl_sync(0xFFFFFFFFu, pages1, at & 31);
        return at < 32 ? lo : hi;
      };
      for (int t = k.a; t < k.b; ++t, ++n) {
        const int key = t * kTile, left = min(k.s.seen - key, kTile), boxes = (left + rows - 1) >> row_bits;
        const int first = key >> p.c.page_bits;
        if (first >= window + 32) {
          window += 32;
          pages0 = pages1;
          pages1 = page_at(window + 32 + lane);
        }
        const int page = page_of(first + min(lane, 15)), within = (key + lane * rows) & (p.c.page_size - 1);
        // 8-bit: the page of this lane's 16 bytes of units, kUnitRows rows
        constexpr int kUnitRows = 512 / D;
        const int unit_row = lane * kUnitRows, unit_page = MX ? page_of(first + (min(unit_row, kTile - 1) >> row_bits)) : 0;
        const int64_t unit_at = MX ? ((static_cast<int64_t>(unit_page) * p.c.heads + k.at.head) * p.c.page_size + ((key + unit_row) & (p.c.page_size - 1))) * (D / 32) : 0;
        const uint32_t found = __ballot_sync(0xFFFFFFFFu, lane < boxes && page >= 0);
#pragma unroll 1
        for (int kv = kv0; kv < kv1; ++kv) {
          const int u = 2 * n + kv;
          const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;
          if constexpr (!MX) {
            const int slot = u % F::STAGES;
            const uint32_t bar = kv_full + 8 * slot, dst = base + F::OFF_KV + slot * F::TILE;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(kv_empty + 8 * slot, ((u / F::STAGES) & 1) ^ 1u, p.w, DEV_ERR_WAIT_PRODUCER));
            if (!ok) break;
            if (elect_one()) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * rows * D * 2));
            __syncwarp();
            if (lane < boxes) tma_load_5d(dst + lane * rows * D * 2, map, bar, 0, 0, 0, within >> 3, page >= 0 ? page * p.page_steps + k.at.head * p.head_steps : -1);
          } else {
            const int slot = u % F::RAWS;
            const uint32_t bar = raw_full + 8 * slot, dst = base + F::OFF_RAW + slot * F::RAW;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(raw_empty + 8 * slot, ((u / F::RAWS) & 1) ^ 1u, p.w, DEV_ERR_WAIT_PRODUCER));
            if (!ok) break;
            // the codes of a page outside the cache are zeros (the copy's fill); its units are not copied
            if (elect_one()) {
              misc->bad[slot] = ~found & ((1u << boxes) - 1u);
              mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * rows * D));
            }
            __syncwarp();
            if (lane < boxes) tma_load_4d(dst + lane * rows * D, map, bar, 0, within, k.at.head, page);
            if (unit_row < left && unit_page >= 0) async_load16(base + F::OFF_UNITS + slot * F::UNITS + 16 * lane, (kv == 0 ? p.c.k_scale : p.c.v_scale) + unit_at);
            async_arrive(bar);
          }
          __syncwarp();
        }
        // (one buffer of queries: this unit's first tile is on its way before the last unit's queries have been read)
        if (ok && F::QBUFS == 1 && kv0 == 0 && t == k.a) load_queries();
        if (!ok) break;
      }
    }
    if (!ok) settle();
  } else if (warp >= F::MMA_WARP) {
    // ---- tensor-core instructions --------------------------------------------------------------------------------------
    // One thread for each tile of rows: with the whole warp walking along and electing a thread for each group of instructions, votes and
    // convergence took some 1700 clocks of an item's 5000 (two tiles of 128 wide heads; 4380 so).
    const int q = warp - F::MMA_WARP;
    if (elect_one()) {
      constexpr uint32_t kScores = idesc_bf16(128, SPREAD ? 128 : 64, false), kValues = idesc_bf16(128, D, true);
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!mbar_try_wait(bar, parity)) ok = mbar_wait_on(bar, parity, p.w, DEV_ERR_WAIT_MMA) && ok;
      };
      // What the loop below needs of a segment, so that it touches the walks at a segment's end only. It is kept short: each of its
      // instructions comes once per item, from wherever the other warps' code has left it.
      struct Part {
        int t, end, lo, hi, filled;  // lo .. hi - 1: what the tile of rows needs
        bool live, fresh;
      };
      auto part_of = [&](Walk<Sequences>& w, Part& x) {
        while (w.live() && w.a >= w.b) w.next();
        x.live = w.live();
        if (!x.live) return;
        x.t = w.a;
        x.end = w.b;
        x.filled = w.filled;
        x.fresh = true;
        const Keys r = w.part_of(q * p.tokens_per_tile, p.tokens_per_tile);
        x.lo = r.lo;
        x.hi = r.hi;
      };
      Walk<Sequences> ahead = k;
      Part s, v;  // the scores' place, one item ahead, and the values'
      part_of(ahead, s);
      part_of(k, v);
      int k_stage = 0, v_stage = F::APART ? F::KEYS : 1;
      uint32_t k_phase = 0, v_phase = 0, q_phase = 0, p_phase = 0, s_slot = 0, v_slot = 0;  // q_phase, p_phase: a bit per buffer or slot
      auto await_keys = [&]() {
        if (s.fresh) {
          const uint32_t buf = NQ == 1 ? s.filled % F::QBUFS : 0;
          wait(q_full + 8 * buf, (q_phase >> buf) & 1u);
          q_phase ^= 1u << buf;
          s.fresh = false;
        }
        wait(kv_full + 8 * k_stage, k_phase);
        tc_fence_after();
      };
      auto await_values = [&]() {
        if (!MX) wait(v_fixed + 8 * v_stage, v_phase);
        wait(kv_full + 8 * v_stage, v_phase);
        tc_fence_after();
      };
      const uint64_t q_desc = smem_desc_sw128(base), k_desc = smem_desc_sw128(base + F::OFF_KV, F::GROUP, 16), v_desc = smem_desc_sw128(base + F::OFF_KV, F::GROUP, 1024);
      auto scores = [&](int half) {  // S = Q K^T
        const int slot = SPREAD ? s_slot : 2 * q + half;
        const uint64_t qd = q_desc + (((NQ == 2 ? q : s.filled % F::QBUFS) * F::TILE) >> 4), kd = k_desc + ((k_stage * F::TILE + half * 8 * F::GROUP) >> 4);
        const uint32_t to = scores_at(slot);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) mma_bf16(to, qd + (((i >> 2) * kPanel + (i & 3) * 32) >> 4), kd + (((i >> 2) * 1024 + (i & 3) * 32) >> 4), kScores, i > 0);
        mma_commit(s_full + 8 * slot);
      };
      auto values = [&](int half, uint32_t phase, bool first) {  // O += P V
        constexpr int STEPS = SPREAD ? 8 : 4;  // of 16 keys
        const int slot = SPREAD ? v_slot : 2 * q + half;
        const uint64_t vd = v_desc + ((v_stage * F::TILE + half * 8 * F::GROUP) >> 4);
        const uint32_t weights = weights_at(slot), o = tmem + 256 + 128 * q, later = first ? 0u : 1u;
        wait(p_ready + 8 * slot, phase);
        tc_fence_after();
        if (!ok) return;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) mma_bf16_ts(o, weights + 8 * i, vd + ((2 * i * F::GROUP) >> 4), kValues, i > 0 ? 1u : later);
        mma_commit(o_done + 8 * slot);
      };
      auto scores_done = [&]() {
        mma_commit(kv_empty + 8 * k_stage);
        k_stage += F::APART ? 1 : 2;
        if (k_stage >= (F::APART ? F::KEYS : F::STAGES)) {
          k_stage -= F::APART ? F::KEYS : F::STAGES;
          k_phase ^= 1;
        }
        s_slot ^= 1;
        if (++s.t == s.end) {
          mma_commit(q_empty + 8 * (NQ == 1 ? s.filled % F::QBUFS : 0));
          ahead.next();
          part_of(ahead, s);
        }
      };
      auto values_done = [&]() {
        mma_commit(kv_empty + 8 * v_stage);
        v_stage += F::APART ? 1 : 2;
        if (v_stage >= F::STAGES) {
          v_stage -= F::APART ? F::STAGES - F::KEYS : F::STAGES;
          v_phase ^= 1;
        }
        v_slot ^= 1;
        if (++v.t == v.end) {
          k.next();
          part_of(k, v);
        }
      };
      // Item by item; the first turn has scores only. Not SPREAD: each half's product with the values, then the next tile's scores
      // over its weights, both in order on the tensor cores. SPREAD: the next tile's scores first, they have a place of their own.
      bool started = false;
      while (ok && (v.live || s.live)) {
        const bool v_turn = started, s_turn = s.live, v_needs = v_turn && v.lo <= v.t && v.t < v.hi, s_needs = s_turn && s.lo <= s.t && s.t < s.hi;
        if (SPREAD) {
          if (s_turn) {
            await_keys();
            if (!ok) break;
            scores(0);
            scores_done();
          }
          if (v_turn) {
            await_values();
            values(0, (p_phase >> v_slot) & 1u, v.t == v.lo);
            if (!ok) break;
            p_phase ^= 1u << v_slot;
            values_done();
          }
        } else {
          if (v_turn) await_values();
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            if (ok && v_needs) values(half, p_phase, half == 0 && v.t == v.lo);
            if (half == 0 && s_turn && ok) await_keys();
            if (ok && s_needs) scores(half);
          }
          if (!ok) break;
          if (v_turn) {
            p_phase ^= v_needs ? 1u : 0u;
            values_done();
          }
          if (s_turn) scores_done();
        }
        started = true;
      }
      mma_commit(bar_final);
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(bar_final, 0))
        if (globaltimer_ns() - t0 > 1000000000ull) {
          atomicOr(p.w.err, DEV_ERR_WAIT_TEARDOWN);
          break;
        }
    }
    __syncwarp();
  } else if (warp >= F::PREP_WARP) {
    // ---- keys and values on their way ----------------------------------------------------------------------------------
    // (one tile of rows: 8-bit keys in the first half of the warps, values in the others)
    constexpr int kGroup = 32 * (MX ? F::GROUP_WARPS : F::PREP_WARPS);
    const int mine = MX && NQ == 1 ? (warp - F::PREP_WARP) / F::GROUP_WARPS : -1, tid = (threadIdx.x - 32 * F::PREP_WARP) % kGroup, rows = min(p.c.page_size, kTile);
    bool ok = true;
    int n = 0;
    for (; ok && k.live(); k.next()) {
      for (int t = k.a; ok && t < k.b; ++t, ++n) {
        const bool edge = k.edge(t);
        const int live = k.s.seen - t * kTile;  // rows that hold keys
        if constexpr (!MX) {
          const int u = 2 * n + 1;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(kv_full + 8 * (u % F::STAGES), (u / F::STAGES) & 1, p.w, DEV_ERR_WAIT_EPILOGUE));
          if (!ok) break;
          uint8_t* v = smem + F::OFF_KV + (u % F::STAGES) * F::TILE;
          bool bad = false;
#pragma unroll 4
          for (int i = tid; (SPREAD || edge) && i < F::PANELS * 1024; i += kGroup) {
            uint4* at = reinterpret_cast<uint4*>(v) + i;
            const uint4 x = *at;
            if ((i / (F::GROUP / 16)) * 8 + ((i >> 3) & 7) >= live) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else if ((not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) != 0u) {
              *at = make_uint4(finite_part(x.x), finite_part(x.y), finite_part(x.z), finite_part(x.w));
              bad = true;
            }
          }
          if (bad) misc->dirty[k.filled & 15] = k.filled;
          if (SPREAD || edge) fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_fixed + 8 * (u % F::STAGES));
        } else {
#pragma unroll 1
          for (int kv = mine < 0 ? 0 : mine; kv <= (mine < 0 ? 1 : mine); ++kv) {
            const int u = 2 * n + kv, raw = u % F::RAWS, slot = F::stage_of(n, kv);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(raw_full + 8 * raw, (u / F::RAWS) & 1, p.w, DEV_ERR_WAIT_EPILOGUE));
            if (!ok) break;
            const uint8_t* codes = smem + F::OFF_RAW + raw * F::RAW;
            const uint8_t* units = smem + F::OFF_UNITS + raw * F::UNITS;
            uint8_t* out = smem + F::OFF_KV + slot * F::TILE;
            const uint32_t lost = misc->bad[raw];
            bool bad = false;
            // A thread's 16 columns (number c) of every kStep-th row; the swizzles' places are the same in all of them. Rows of 128: eight
            // lanes take four c of rows r and r ^ 5, which meet in no bank, neither in the codes nor in the panels.
            constexpr int kLanes = D / 16, kStep = kGroup / kLanes, kRows = 128 / kStep;
            const int pair = (tid >> 4) & 3, row0 = D == 128 ? 8 * (tid >> 6) + (tid & 4 ? pair ^ 5 : pair) : tid / kLanes;
            const int c = D == 128 ? (tid & 3) + ((tid >> 1) & 4) : tid % kLanes, at = row0 * kLanes + (D == 128 ? c ^ (row0 & 7) : c);
            uint4 x[kRows];
            uint32_t unit[kRows], largest = 0u;
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
              x[j] = reinterpret_cast<const uint4*>(codes)[at + kGroup * j];
              unit[j] = units[(row0 + j * kStep) * (D / 32) + c / 2];
            }
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(kv_empty + 8 * slot, F::phase_of(n, kv) ^ 1u, p.w, DEV_ERR_WAIT_EPILOGUE));
            if (!ok) break;
            uint8_t* panel = out + (row0 >> 3) * F::GROUP + (c >> 2) * 1024 + (row0 & 7) * 128;
            uint4* first = reinterpret_cast<uint4*>(panel + (((2 * (c & 3)) ^ (row0 & 7)) << 4));
            uint4* second = reinterpret_cast<uint4*>(panel + (((2 * (c & 3) + 1) ^ (row0 & 7)) << 4));
            auto store = [&](int j, const uint32_t (&y)[8]) {
              first[j * (kStep / 8) * (F::GROUP / 16)] = make_uint4(y[0], y[1], y[2], y[3]);
              second[j * (kStep / 8) * (F::GROUP / 16)] = make_uint4(y[4], y[5], y[6], y[7]);
            };
#pragma unroll
            for (int j = 0; j < kRows; ++j) largest = max(largest, unit[j]);
            if (largest < 135u && lost == 0u && (kv == 0 || live >= kTile)) {  // 2^(unit - 127) 2^120 is a bf16, and all values are finite
#pragma unroll
              for (int j = 0; j < kRows; ++j) {
                uint32_t y[8];
                decode16(x[j], bf16_pair((unit[j] + 120u) << 7), y);
                store(j, y);
              }
            } else {
#pragma unroll 1
              for (int j = 0; j < kRows; ++j) {
                const int row = row0 + j * kStep;
                const uint32_t byte = units[row * (D / 32) + c / 2];
                uint32_t y[8], any = 0u;
                decode16(reinterpret_cast<const uint4*>(codes)[at + kGroup * j], bf16_pair(0x7B80u), y);  // in two factors
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  y[e] = times(y[e], bf16_pair(byte == 255u ? 0x7FC0u : byte == 0u ? 0x0040u : byte << 7));
                  if ((lost >> (row / rows) & 1u) || (kv == 1 && row >= live)) y[e] = 0u;
                  any |= not_finite(y[e]);
                }
                if (kv == 1 && (edge || SPREAD) && any != 0u) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = finite_part(y[e]);
                  bad = true;
                }
                store(j, y);
              }
            }
            if (bad) misc->dirty[k.filled & 15] = k.filled;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(kv_full + 8 * slot);
              mbar_arrive(raw_empty + 8 * raw);
            }
          }
        }
      }
    }
  } else if (warp < 4 * NQ) {
    // ---- weights: a thread per row; SPREAD: a thread per row and quarter of a tile's keys ------------------------------
    const int q = warp >> 2, row = SPREAD ? lane : threadIdx.x & 127, key0 = SPREAD ? 32 * warp : 0;
    constexpr int HALVES = SPREAD ? 1 : 2, KEYS = SPREAD ? 32 : 64;  // steps of a tile, a thread's keys of a step
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t o_at = tmem + lanes + 256 + 128 * q;
    const int token = (row * p.group_inverse) >> 16;
    // (a score of +infinity: the reference stays finite, so that the weight and the sum become infinite and not NaN)
    const float c2 = p.c2, slack = fminf(kSlack / c2, 3.0e38f), highest = fminf(3.0e38f / c2, 3.0e38f);
    bool ok = true;
    int n = 0;  // tiles of this warpgroup so far
    // A step's slot, and its barriers' phase. When the scores of a step are there, the product with the values of the last step but one is
    // done; of the last step's the barrier tells (the other of two, so that neither can be a phase ahead of what is asked).
    auto slot_of = [&](int tile, int half) { return SPREAD ? tile & 1 : 2 * q + half; };
    auto phase_of = [&](int tile) { return static_cast<uint32_t>(SPREAD ? tile >> 1 : tile) & 1u; };
    auto values_done = [&](int tile, int half) { return mbar_wait(o_done + 8 * slot_of(tile, half), phase_of(tile), p.w, DEV_ERR_WAIT_EPILOGUE); };
    if constexpr (SPREAD) {  // the weights that this warp's copy of the rows gives to the other warps' keys
      uint32_t none[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) none[e] = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) tmem_st32(tmem + lanes + 384 + 32 * e, none);
      tmem_st_wait();
    }
    for (; k.live(); k.next()) {
      const int i0 = k.at.block * per + q * p.tokens_per_tile, i = i0 + token;
      if (i0 >= k.s.n) continue;
      const bool valid = token < p.tokens_per_tile && i < k.s.n;
      Keys mine{0, 0};
      if (valid) mine = keys_of(k.s, i, p.a.window);
      const Keys part = k.part_of(q * p.tokens_per_tile, p.tokens_per_tile);
      const bool any = __any_sync(0xFFFFFFFFu, valid);
      float m = -INFINITY, limit = -INFINITY, l = 0.0f;
      for (int t = part.lo; t < part.hi; ++t, ++n) {
#pragma unroll 1
        for (int half = 0; half < HALVES; ++half) {
          const int slot = slot_of(n, half);
          const uint32_t s_at = scores_at(slot) + lanes + key0, w_at = weights_at(slot) + lanes + key0 / 2;
          ok = ok && mbar_wait(s_full + 8 * slot, phase_of(n), p.w, DEV_ERR_WAIT_EPILOGUE);
          __syncwarp();
          tc_fence_after();
          if (any) {
            uint32_t r0[32], r1[32];
            tmem_ld32(s_at, r0);
            if constexpr (!SPREAD) tmem_ld32(s_at + 32, r1);
            tmem_ld_wait();
            reg_fence(r0);
            reg_fence(r1);
            const int key = t * kTile + 64 * half + key0;
            if (p.flip || !__all_sync(0xFFFFFFFFu, !valid || (mine.lo <= key && key + KEYS <= mine.hi))) {
              const int lo = mine.lo - key;
              const uint32_t width = static_cast<uint32_t>(most(mine.hi - mine.lo, 0)), sign = p.flip ? 0x80000000u : 0u;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                r0[e] = static_cast<uint32_t>(e - lo) < width ? r0[e] ^ sign : 0xFF800000u;
                if constexpr (!SPREAD) r1[e] = static_cast<uint32_t>(e + 32 - lo) < width ? r1[e] ^ sign : 0xFF800000u;
              }
            }
            float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              top = max3(top, __uint_as_float(r0[e]), __uint_as_float(r0[e + 1]));
              top1 = max3(top1, __uint_as_float(r0[e + 2]), __uint_as_float(r0[e + 3]));
            }
            if constexpr (!SPREAD) {
              float top2 = -INFINITY, top3 = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                top2 = max3(top2, __uint_as_float(r1[e]), __uint_as_float(r1[e + 1]));
                top3 = max3(top3, __uint_as_float(r1[e + 2]), __uint_as_float(r1[e + 3]));
              }
              top = max3(top, top2, top3);
            }
            top = fmaxf(top, top1);
            const bool move = valid && top > limit;
            if (__any_sync(0xFFFFFFFFu, move)) {  // the reference moves
              const float to = move ? fminf(top, highest) : m;
              if (t > part.lo || half > 0) {
                const float f = move ? exp2_of((m - to) * c2) : 1.0f;
                l *= f;
                ok = ok && (half > 0 ? values_done(n, 0) : values_done(n - 1, HALVES - 1));
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                  uint32_t x[16];
                  tmem_ld16(o_at + d, x);
                  tmem_ld_wait();
                  reg_fence(x);
#pragma unroll
                  for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                  tmem_st16(o_at + d, x);
                }
              }
              m = to;
              if (move) limit = top + slack;
            }
            const uint64_t c = both(c2), shift = both(m == -INFINITY ? 0.0f : -(m * c2));
            uint64_t sum0 = 0, sum1 = 0;
            auto weigh = [&](uint32_t (&r)[32], uint32_t at) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 x = split(fma2(pair(r[2 * e], r[2 * e + 1]), c, shift));
                const float a = exp2_of(x.x), b = exp2_of(x.y);
                const uint64_t ab = pair(__float_as_uint(a), __float_as_uint(b));
                if (e & 1)
                  sum1 = add2(sum1, ab);
                else
                  sum0 = add2(sum0, ab);
                w[e] = heads::pack(a, b);
              }
              tmem_st16(at, w);
            };
            weigh(r0, w_at);
            if constexpr (!SPREAD) weigh(r1, w_at + 16);
            const float2 s = split(add2(sum0, sum1));
            l += s.x + s.y;
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready + 8 * slot);
          __syncwarp();
        }
      }
      // ---- the unit's end, or this CTA's part's ------------------------------------------------------------------------
      const bool some = part.lo < part.hi, alone = k.first() && k.last();
      const int64_t unit0 = k.at.item - k.at.off;
      const int c0 = alone ? 0 : cta_of(total, unit0, runs), c1 = alone ? 0 : least(cta_of(total, unit0 + k.items - 1, runs), runs - 1);  // (lengths that changed under the call)
      char* to = alone ? nullptr : part_at<D, NQ>(p, c0, blockIdx.x, q);
      const int rows = least(k.s.n - i0, p.tokens_per_tile) * p.group;  // of this tile
      auto set_lse = [&](int r, float reference, float sum) { put_lse(p, static_cast<int64_t>(k.s.first) + i0, k.at.head * p.group, r, reference, sum); };
      // where this thread puts elements of its row (SPREAD: of the row that it adds up), done or as they are
      const int own = SPREAD ? static_cast<int>(threadIdx.x) >> 2 : row, block = own & ~31, across = least(rows - block, 32);
      char* const place = own >= rows ? nullptr
                          : alone     ? reinterpret_cast<char*>(row_of(p, static_cast<int64_t>(k.s.first) + i0, k.at.head * p.group, own))
                                      : to + 1024 + 16 * (block * (D / 4) + own - block);
      auto put8 = [&](int d, const float (&y)[8], float sum, float inv) {
        if (alone) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = sum == 0.0f ? 0u : heads::pack(y[2 * j] * inv, y[2 * j + 1] * inv);
          *reinterpret_cast<uint4*>(place + 2 * d) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          float4* o = reinterpret_cast<float4*>(place) + (d / 4) * across;
          __stcg(o, make_float4(y[0], y[1], y[2], y[3]));
          __stcg(o + across, make_float4(y[4], y[5], y[6], y[7]));
        }
      };
      auto add_unusual = [&](int d, float (&x)[8]) {  // what was taken out of the values that this thread's row sees
        for (int t = part.lo; t < part.hi; ++t) {
          if (!SPREAD && !k.edge(t)) continue;
          for (int j = most(mine.lo, t * kTile + key0); j < least(mine.hi, t * kTile + (SPREAD ? key0 + 32 : kTile)); ++j) {
            const int page = __ldg(p.b.page_table + k.at.seq * p.b.ld_table + (j >> p.c.page_bits));
            if (page < 0 || page >= p.c.pages) continue;
            const int at = j & (p.c.page_size - 1);
            const int64_t v_row = page * p.c.page_stride + k.at.head * p.c.head_stride + at * p.c.token_stride;
            const int64_t unit = ((static_cast<int64_t>(page) * p.c.heads + k.at.head) * p.c.page_size + at) * (D / 32);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += unusual<MX, D>(p, v_row, unit, d + e);
          }
        }
      };
      if (some && any) {
        ok = ok && values_done(n - 1, HALVES - 1);
        __syncwarp();
        tc_fence_after();
      }
      const bool dirty = some && *reinterpret_cast<volatile int*>(&misc->dirty[k.filled & 15]) == k.filled;
      if constexpr (SPREAD) {
        // the four warps' copies of a row, each over its own keys, are brought to one reference and added
        float2* stats = reinterpret_cast<float2*>(smem + F::OFF_STATS);
        float4* share = reinterpret_cast<float4*>(smem + (F::SHARE != 0 ? F::OFF_SHARE : (k.filled & 1) * F::TILE));  // (the unit's queries, which nothing reads any more)
        stats[threadIdx.x] = make_float2(m * c2, l);
        bar_sync(1, 128);
        auto joined = [&](int r) {
          float2 s = make_float2(-INFINITY, 0.0f);
#pragma unroll
          for (int w = 0; w < 4; ++w) s.x = fmaxf(s.x, stats[32 * w + r].x);
          if (s.x == -INFINITY) s.x = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) s.y = fmaf(exp2_of(stats[32 * w + r].x - s.x), stats[32 * w + r].y, s.y);
          return s;
        };
        const float f = exp2_of(m * c2 - joined(lane).x);
        const int r = threadIdx.x >> 2, e0 = threadIdx.x & 3;  // a row and 8 of 32 columns
        const float2 s = joined(r);
        const float inv = inverse_of(s.y);
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          if (some) {
            uint32_t x[32];
            tmem_ld32(o_at + d, x);
            tmem_ld_wait();
            reg_fence(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float y[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(x[8 * e + j]) * f;
              if (dirty && valid) add_unusual(d + 8 * e, y);
              share[threadIdx.x * 8 + ((2 * e) ^ (lane & 7))] = make_float4(y[0], y[1], y[2], y[3]);
              share[threadIdx.x * 8 + ((2 * e + 1) ^ (lane & 7))] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
          bar_sync(1, 128);
          if (r < rows) {
            float y[8] = {};
            if (some) {
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const float4 a = share[(32 * w + r) * 8 + ((2 * e0) ^ (r & 7))], b = share[(32 * w + r) * 8 + ((2 * e0 + 1) ^ (r & 7))];
                y[0] += a.x, y[1] += a.y, y[2] += a.z, y[3] += a.w, y[4] += b.x, y[5] += b.y, y[6] += b.z, y[7] += b.w;
              }
            }
            put8(d + 8 * e0, y, s.y, inv);
          }
          bar_sync(1, 128);
        }
        if (e0 == 0 && r < rows) {
          if (alone)
            set_lse(r, s.x, s.y);
          else
            __stcg(reinterpret_cast<float2*>(to) + r, make_float2(s.y == 0.0f ? -INFINITY : s.x, s.y));
        }
        if (F::SHARE == 0 && some) {
          fence_proxy_async_smem();
          bar_sync(1, 128);
          if (threadIdx.x == 0) mbar_arrive(q_empty + 8 * (k.filled & 1));
        }
      } else if (any) {
        const float inv = inverse_of(l);
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t x[32];
          if (some) {
            tmem_ld32(o_at + d, x);
            tmem_ld_wait();
            reg_fence(x);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0u;
          }
          if (!valid) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(x[8 * e + j]);
            if (dirty) add_unusual(d + 8 * e, y);
            put8(d + 8 * e, y, l, inv);
          }
        }
        if (valid && alone) set_lse(row, m * c2, l);
        if (valid && !alone) __stcg(reinterpret_cast<float2*>(to) + row, make_float2(m * c2, l));
      }
      tc_fence_before();
      if (!alone) {
        __threadfence();
        bar_sync(1 + q, 128);
        if ((threadIdx.x & 127) == 0 && atomicAdd(p.counters + 2 * c0 + q, 1u) == static_cast<unsigned>(c1 - c0)) {
          p.counters[2 * c0 + q] = 0u;
          misc->join[2 * q + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)] = Join{static_cast<int64_t>(k.s.first) + i0, k.at.head * p.group, rows, c0, c1};
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == F::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  uint32_t phase = 0;
  bool joined = true;
#pragma unroll 1
  for (int i = 0; i < 2 * NQ && joined; ++i)
    if (misc->join[i].rows > 0) joined = join_parts<D, NQ, F::THREADS>(p, misc->join[i], i >> 1, smem, reinterpret_cast<float*>(smem + F::OFF_STATS), bar_join, phase);
  if (!joined) settle();  // (copies may be in flight)
}

int ctas() { return min(num_sms(), kMaxCtas); }

// Which form, by the rows that a sequence has for a cache head on average (the lengths are on the device). Measured with 64 sequences
// over 4096 keys, 8 heads, D 128, in us:
//   rows              4     16     32     36     64    128    132    192    256
//   32, four times  174    177    179    332    337                              (8-bit: 147  149  151  279  281)
//   one tile        175    179    183    183    186    193    349    356    359
//   two tiles       177    181    183    185    188    193    219    234    243  (8-bit: 175  178  178  179  180  183  227  234  243)
// (D 64, 4 rows: 94, 133 and 148, 8-bit 98 and 156; one token over 100 keys, D 64: 7.0, 7.4 and 8.0.) So up to 32 rows: a tile of 32, each of the
// four warps of weights with its own quarter of the keys. Above: two tiles, but one in bf16 where units do not fill it (8-bit caches
// have no such form: with earlier stages it took 221 to 251 us for 4 to 128 rows, with the present ones it has not been measured).
// What an average does not see is a batch of many short sequences and a long one: 255 single tokens over 4096 keys and a chunk of 1793 over
// 16384 (32 rows on average) take 2100 us in the first form, of which the chunk's blocks of 8 tokens are two thirds, and 1035 in the second;
// by themselves the tokens take 632 and the chunk, in the third form, 337. Calls of their own for long chunks are faster there.
bool spread(const Attention& a, const Cache& c, const Batch& b) {
  const int64_t group = a.q_heads / c.heads;
  return group <= 32 && b.tokens * group <= static_cast<int64_t>(b.seqs) * 32;
}
bool two_tiles(const Attention& a, const Cache& c, const Batch& b) {
  return !spread(a, c, b) && (c.mx || b.tokens * (a.q_heads / c.heads) > static_cast<int64_t>(b.seqs) * kTile);
}

// A bf16 cache's pages and heads as one dimension of its tensor maps, at the strides' common part.
struct Steps {
  int64_t unit, page, head, all;
};
Steps steps_of(const Cache& c) {
  const int64_t ps = c.pages > 1 ? c.page_stride : 0, hs = c.heads > 1 ? c.head_stride : 0, both = std::gcd(ps, hs), unit = both != 0 ? both : c.token_stride;
  return Steps{unit, ps / unit, hs / unit, (static_cast<int64_t>(max(c.pages, 1)) - 1) * (ps / unit) + (c.heads - 1) * (hs / unit) + 1};
}

int tokens_of_tile(const Attention& a, const Cache& c, const Batch& b) { return (spread(a, c, b) ? 32 : kTile) / (a.q_heads / c.heads); }
// (a cache without pages holds nothing, and the tensor maps need an address)
int reach_of(const Cache& c, const Batch& b) { return static_cast<int>(min(c.pages > 0 ? static_cast<int64_t>(b.table_width) << c.page_bits : 0, int64_t{0x7FFFFF00})); }

template <int D, bool MX, int NQ, bool SPREAD>
cudaError_t launch_form(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Params& p, cudaStream_t stream) {
  using F = Form<D, MX, NQ, SPREAD>;
  auto* kernel = paged_attention_kernel<D, MX, NQ, SPREAD>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas()), dim3(F::THREADS), F::SMEM, stream, q, k, v, p);
}

}  // namespace

const char* paged_attention_refusal(const Attention& a, const Cache& c, const Batch& b) {
  if (!c.mx && steps_of(c).all > 0x7FFFFFFF) return "pages and heads of the cache lie at strides whose common part is too small";
  const int64_t limit = int64_t{1} << 39;  // tensor maps' strides are below 2^40 bytes, the widest one here 16 tokens of bf16
  auto far = [&](int64_t n, int64_t stride) { return n > 1 && stride >= limit; };
  if (c.token_stride >= limit / 16 || far(c.heads, c.head_stride) || far(c.pages, c.page_stride) || far(b.tokens, a.ld_q) || far(a.q_heads, a.hs_q)) return "a stride of 2^39 elements or more (2^35 between a cache's tokens)";
  // tiles of keys over blocks of rows, counted in 32 bits per sequence and in 64 over all of them (times the CTAs)
  const int64_t per = (two_tiles(a, c, b) ? 2 : 1) * tokens_of_tile(a, c, b);
  const __int128 tiles = static_cast<__int128>(b.tokens / per + 1) * (reach_of(c, b) / kTile + 1);
  if (tiles >= 0xFFFFFFFF || tiles * max(b.seqs, 1) * c.heads >= (static_cast<__int128>(1) << 54)) return "more tokens over a longer table than a call counts";
  return nullptr;
}

int64_t paged_attention_workspace_bytes(const Attention& a, const Cache& c, const Batch& b) {
  return kCounterBytes + static_cast<int64_t>(ctas()) * 2 * (two_tiles(a, c, b) ? 2 : 1) * 128 * (c.head_dim + 2) * 4;
}

cudaError_t launch_paged_attention(const Attention& a, const Cache& c, const Batch& b, void* ws, cudaStream_t stream, const char** why) {
  Params p{};
  p.a = a;
  p.c = c;
  p.b = b;
  p.group = a.q_heads / c.heads;
  p.group_inverse = (65536 + p.group - 1) / p.group;
  const bool two = two_tiles(a, c, b), four = spread(a, c, b);
  p.tokens_per_tile = tokens_of_tile(a, c, b);
  p.capacity = reach_of(c, b);
  // scale 0: every weight is 1, and -infinity times it stays -infinity
  p.c2 = max(std::fabs(a.scale) * kLog2e, 1.0e-44f);
  p.flip = a.scale < 0.0f;
  p.counters = static_cast<unsigned*>(ws);
  p.parts = static_cast<char*>(ws) + kCounterBytes;
  p.w = wait_ctl();
  if (p.w.err == nullptr) {
    *why = "device error word unavailable";
    return cudaErrorInvalidDevice;
  }
  const uint64_t D = static_cast<uint64_t>(c.head_dim), row = 2 * D;
  CUtensorMap mq, mk, mv;
  auto or_row = [](int64_t n, int64_t stride_bytes, uint64_t otherwise) { return n > 1 ? static_cast<uint64_t>(stride_bytes) : otherwise; };
  const uint64_t q_dims[3] = {D, static_cast<uint64_t>(a.q_heads), static_cast<uint64_t>(b.tokens)};
  const uint64_t q_strides[2] = {or_row(a.q_heads, 2 * a.hs_q, row), or_row(b.tokens, 2 * a.ld_q, row)};
  const uint32_t q_box[3] = {64, static_cast<uint32_t>(p.group), static_cast<uint32_t>(p.tokens_per_tile)};
  const uint64_t pages = static_cast<uint64_t>(max(c.pages, 1));
  const void* k = c.pages > 0 ? c.k : a.q;
  const void* v = c.pages > 0 ? c.v : a.q;
  bool made = encode_tmap_nd(&mq, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q_dims, q_strides, q_box, 128);
  const uint32_t rows = static_cast<uint32_t>(min(c.page_size, kTile));
  if (c.mx) {
    const uint64_t dims[4] = {D, static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(c.heads), pages};
    const uint64_t strides[3] = {static_cast<uint64_t>(c.token_stride), or_row(c.heads, c.head_stride, D), or_row(c.pages, c.page_stride, D)};
    const uint32_t box[4] = {static_cast<uint32_t>(D), rows, 1, 1};
    made = made && encode_tmap_nd(&mk, k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, dims, strides, box, D == 128 ? 128 : 0) &&
           encode_tmap_nd(&mv, v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, dims, strides, box, D == 128 ? 128 : 0);
  } else {
    // a tile's rows by groups of 8, both panels of a group one after the other: with a box for each panel the two halves of
    // a row's 256 bytes were fetched far apart (64 tokens over 4096: 1.0 TB/s with 128 rows a box, 5.8 with 16, 6.1 so)
    const Steps steps = steps_of(c);
    p.page_steps = static_cast<int>(steps.page);
    p.head_steps = static_cast<int>(steps.head);
    const uint64_t dims[5] = {64, 8, D / 64, static_cast<uint64_t>(c.page_size / 8), static_cast<uint64_t>(steps.all)};
    const uint64_t strides[4] = {static_cast<uint64_t>(2 * c.token_stride), 128, static_cast<uint64_t>(16 * c.token_stride), static_cast<uint64_t>(2 * steps.unit)};
    const uint32_t box[5] = {64, 8, static_cast<uint32_t>(D / 64), rows / 8, 1};
    made = made && encode_tmap_nd(&mk, k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, dims, strides, box, 128) && encode_tmap_nd(&mv, v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, dims, strides, box, 128);
  }
  if (!made) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
#define FP8GB_FORM(D, MX, NQ, SPREAD) launch_form<D, MX, NQ, SPREAD>(mq, mk, mv, p, stream)
  if (c.mx) {
    if (c.head_dim == 64) return four ? FP8GB_FORM(64, true, 1, true) : FP8GB_FORM(64, true, 2, false);
    return four ? FP8GB_FORM(128, true, 1, true) : FP8GB_FORM(128, true, 2, false);
  }
  if (c.head_dim == 64) return two ? FP8GB_FORM(64, false, 2, false) : four ? FP8GB_FORM(64, false, 1, true) : FP8GB_FORM(64, false, 1, false);
  return two ? FP8GB_FORM(128, false, 2, false) : four ? FP8GB_FORM(128, false, 1, true) : FP8GB_FORM(128, false, 1, false);
#undef FP8GB_FORM
}

}  // namespace fp8gb
