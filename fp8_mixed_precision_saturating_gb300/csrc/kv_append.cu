// kv_append.cu -- queries, keys and values of new tokens from the projection's rows: queries and keys normed and turned
// (heads.cuh), keys and values into the slots of a paged cache, as bf16 or as E4M3 with a power of two per 32 elements.
//
// What bounds it: memory, each element in once and out once; for a few tokens the chain of loads (the token's sequence, its length, its page,
// then the rows). A warp takes a token and a run of its heads, so that this chain and the angles are paid once per run.
// Measured, 32 + 8 + 8 heads of 128, bf16 cache: a prompt of 8192 tokens 37.3 us, 5.4 TB/s (the rotation alone runs at 6.35: each warp waits for its chain
// once; runs of 32 heads 40; 8 rows at once half as fast); one token of 64 sequences 3.7 us, the launch and the chain.
#include "heads.cuh"

namespace fp8gb {
namespace {

using namespace heads;

// Small CTAs: a warp's slot is free again when its CTA's last warp is done (a prompt of 8192 tokens, items in the tokens'
// order: 39.0 us; CTAs of 128 threads 39.5, of 256 42.6).
constexpr int kThreads = 64, kWarps = kThreads / 32;

struct Args {
  Turn t;
  Heads part[3];  // queries, keys, values
  Cache c;
  Batch b;
  int per;         // heads of one item
  int first[3];    // items of a token before each part's
  int items;
  int64_t total;
};

// A group's power of two and the factor its elements take, from its largest magnitude (NaN: any NaN among them).
struct Unit {
  uint32_t byte;
  float factor;
};
__device__ __forceinline__ Unit unit_of(float a) {
  Unit u;
  if (a != a) {
    u.byte = 0xFFu;
    u.factor = 0.0f;
    return u;
  }
  a = fminf(a, 3.3895314e38f);  // an infinity counts as the largest finite bf16
  const uint32_t b = __float_as_uint(a);
  // a = 1.m 2^(x - 127); 448 = 1.75 * 2^8
  int e = static_cast<int>(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = b == 0u ? 0 : max(e, -127);
  u.byte = static_cast<uint32_t>(e + 127);
  u.factor = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // e <= 120, and 2^127 for the least
  return u;
}
__device__ __forceinline__ float nan_max(float a, float b) { return a != a || b != b ? __int_as_float(0x7FFFFFFF) : fmaxf(a, b); }
__device__ __forceinline__ uint32_t codes2(float lo, float hi, const Unit& u) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi * u.factor), "f"(lo * u.factor));
  return u.byte == 0xFFu ? 0u : r;
}

// The place of a token's rows in the cache: the page's offset and the token's, or none.
struct Slot {
  bool in;
  int64_t page;
  int at;
};
__device__ __forceinline__ Slot slot_of(const Place& at, const Cache& c, const Batch& b) {
  Slot s{false, 0, 0};
  if (at.seq < 0 || at.pos < 0 || at.pos >= static_cast<int64_t>(b.table_width) << c.page_bits) return s;
  const int page = __ldg(b.page_table + at.seq * b.ld_table + (at.pos >> c.page_bits));
  s.in = page >= 0 && page < c.pages;
  s.page = page;
  s.at = static_cast<int>(at.pos & (c.page_size - 1));
  return s;
}
__device__ __forceinline__ int64_t row_at(const Slot& s, const Cache& c, int h) {
  return s.page * c.page_stride + h * c.head_stride + s.at * c.token_stride;
}
__device__ __forceinline__ int64_t unit_at(const Slot& s, const Cache& c, int h) {
  return ((s.page * c.heads + h) * c.page_size + s.at) * (c.head_dim / 32);
}

// All tokens' queries come first, then the keys, then the values: the warps of a CTA have the same work (in the order of the tokens: 39.0 us).
struct Item {
  int64_t token;
  int part, h0, h1;
};
__device__ __forceinline__ Item item_of(int64_t i, const Args& g) {
  Item m;
  m.part = i >= g.b.tokens * g.first[2] ? 2 : i >= g.b.tokens * g.first[1] ? 1 : 0;
  i -= g.b.tokens * g.first[m.part];
  const int items = (m.part == 2 ? g.items : g.first[m.part + 1]) - g.first[m.part];
  m.token = items == 1 ? i : i >> 32 == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(items) : i / items;
  m.h0 = static_cast<int>(i - m.token * items) * g.per;
  m.h1 = min(m.h0 + g.per, g.part[m.part].n);
  return m;
}

// 8 consecutive elements of a row into the 8-bit cache: a unit is 4 lanes' worth.
__device__ __forceinline__ void store_mx(const float (&x)[8], bool live, int d, uint8_t* codes, uint8_t* units) {
  float a = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = nan_max(a, fabsf(x[k]));
  a = nan_max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
  a = nan_max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
  const Unit u = unit_of(a);
  if (!live) return;
  uint2 w;
  w.x = codes2(x[0], x[1], u) | (codes2(x[2], x[3], u) << 16);
  w.y = codes2(x[4], x[5], u) | (codes2(x[6], x[7], u) << 16);
  *reinterpret_cast<uint2*>(codes + d) = w;
  if ((d & 31) == 0) units[d >> 5] = static_cast<uint8_t>(u.byte);
}

template <bool INTER, int LPR, bool MX, bool PARTIAL>
__global__ void __launch_bounds__(kThreads, 12) kv_append_kernel(const __grid_constant__ Args g) {
  constexpr int RPW = 32 / LPR, U = 4;
  // keys on their way into 8 bits: a warp's rows, turned, to be read 8 consecutive elements a lane
  __shared__ __align__(16) float share[MX ? kWarps : 1][MX ? RPW : 1][MX ? LPR * 8 : 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR, l = lane % LPR;
  const Lane a = lane_of<INTER>(l, g.t.head_dim, g.t.rot_dims);
  pdl_wait();
  pdl_trigger();
  const int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kWarps + warp;
  if (i >= g.total) return;
  const Item m = item_of(i, g);
  const Heads& p = g.part[m.part];
  const bf16* in = static_cast<const bf16*>(p.in) + m.token * p.ld_in;
  if (m.part == 2) {  // values: as they are
    uint4 raw[U];
    auto load = [&](int h0) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = h0 + j * RPW + sub;
        raw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (a.in && h < m.h1) {
          const uint2* q = reinterpret_cast<const uint2*>(in + h * p.hs_in + 8 * l);
          const uint2 x = __ldcs(q), y = __ldcs(q + 1);
          raw[j] = make_uint4(x.x, x.y, y.x, y.y);
        }
      }
    };
    load(m.h0);
    const Slot at = slot_of(place_of(m.token, g.b, lane), g.c, g.b);
    if (!at.in) return;
#pragma unroll 1
    for (int h0 = m.h0; h0 < m.h1; h0 += U * RPW) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = h0 + j * RPW + sub;
        const bool live = a.in && h < m.h1;
        const int64_t row = row_at(at, g.c, h);
        if constexpr (MX) {
          const float x[8] = {lo_of(raw[j].x), hi_of(raw[j].x), lo_of(raw[j].y), hi_of(raw[j].y), lo_of(raw[j].z), hi_of(raw[j].z), lo_of(raw[j].w), hi_of(raw[j].w)};
          store_mx(x, live, 8 * l, static_cast<uint8_t*>(g.c.v) + row, g.c.v_scale + unit_at(at, g.c, h));
        } else if (live) {
          *reinterpret_cast<uint4*>(static_cast<bf16*>(g.c.v) + row + 8 * l) = raw[j];
        }
      }
      if (h0 + U * RPW < m.h1) load(h0 + U * RPW);
    }
    return;
  }
  // (lanes past the head hold zeros; a row past the last one is the last one again, and not stored)
  Raw<bf16, INTER> raw[U], next[U] = {};
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (a.in) next[j].load(in + min(h0 + j * RPW + sub, m.h1 - 1) * p.hs_in, a.o0, a.o1);
  };
  load(m.h0);
  const Place where = place_of(m.token, g.b, lane);
  const Slot at = slot_of(where, g.c, g.b);
  if (where.seq < 0 || (m.part == 1 && !at.in)) return;  // a row of nobody; a key without a place
  const int32_t pos = g.t.pos != nullptr ? __ldg(g.t.pos + m.token) : static_cast<int32_t>(where.pos);
  float c[4], s[4], wu[4], wv[4];
  angles<LPR>(a, g.t.turns, g.t.rot_dims, pos, g.t.amplitude, c, s);
  weights<INTER>(a, p.w, wu, wv);
  const Factors f = factors(c, s, wu, wv);
  const float inv_dim = 1.0f / static_cast<float>(g.t.head_dim);
  bf16* out = m.part == 0 ? static_cast<bf16*>(p.out) + m.token * p.ld_out : nullptr;
#pragma unroll 1
  for (int h0 = m.h0; h0 < m.h1; h0 += U * RPW) {
#pragma unroll
    for (int j = 0; j < U; ++j) raw[j] = next[j];
    if (h0 + U * RPW < m.h1) load(h0 + U * RPW);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      Pair u[2], v[2], yu[2], yv[2];
      const int h = h0 + j * RPW + sub;
      const bool live = a.in && h < m.h1;
      raw[j].get(u, v);
      if (g.t.norm)
        turn<LPR, true, INTER, PARTIAL>(a, f, inv_dim, g.t.eps, u, v, yu, yv);
      else
        turn<LPR, false, INTER, PARTIAL>(a, f, inv_dim, g.t.eps, u, v, yu, yv);
      if (m.part == 0) {
        if (live) Raw<bf16, INTER>::put(out + h * p.hs_out, a.o0, a.o1, yu, yv);
      } else if constexpr (MX) {
        float* row = share[warp][sub];
        if (a.in) put_shared<INTER>(row, a.o0, a.o1, yu, yv);
        __syncwarp();
        float x[8] = {};
        if (a.in) {
          const float4 x0 = *reinterpret_cast<const float4*>(row + 8 * l), x1 = *reinterpret_cast<const float4*>(row + 8 * l + 4);
          x[0] = x0.x, x[1] = x0.y, x[2] = x0.z, x[3] = x0.w, x[4] = x1.x, x[5] = x1.y, x[6] = x1.z, x[7] = x1.w;
        }
        store_mx(x, live, 8 * l, static_cast<uint8_t*>(g.c.k) + row_at(at, g.c, h), g.c.k_scale + unit_at(at, g.c, h));
        __syncwarp();
      } else if (live) {
        Raw<bf16, INTER>::put(static_cast<bf16*>(g.c.k) + row_at(at, g.c, h), a.o0, a.o1, yu, yv);
      }
    }
  }
}

// Rows of single elements, a warp each. (A prompt of 8192 tokens of 32 + 8 + 8 heads of 128, 60 elements turning: 193 us, in 8 bits 215; without the
// bounds 242 and 258, with registers for fewer CTAs.)
template <bool MX>
__global__ void __launch_bounds__(kThreads, MX ? 10 : 14) kv_append_any_kernel(const __grid_constant__ Args g) {
  __shared__ float share[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = g.t.head_dim, R = g.t.rot_dims;
  pdl_wait();
  pdl_trigger();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < g.total; i += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Item m = item_of(i, g);
    const Heads& p = g.part[m.part];
    const Place where = place_of(m.token, g.b, lane);
    const Slot at = slot_of(where, g.c, g.b);
    if (where.seq < 0 || (m.part != 0 && !at.in)) continue;
    const int32_t pos = g.t.pos != nullptr ? __ldg(g.t.pos + m.token) : static_cast<int32_t>(where.pos);
    for (int h = m.h0; h < m.h1; ++h) {
      const bf16* in = static_cast<const bf16*>(p.in) + m.token * p.ld_in + h * p.hs_in;
      float x[8], q = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = lane + 32 * k;
        x[k] = d < D ? element(in + d) : 0.0f;
        q = fmaf(x[k], x[k], q);
      }
      if (m.part != 2) {
        const float r = g.t.norm ? rsqrtf(fmaf(row_sum<32>(q), 1.0f / static_cast<float>(D), g.t.eps)) : 1.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int d = lane + 32 * k;
          x[k] *= r * (d < D && p.w != nullptr ? __ldg(p.w + d) : 1.0f);
          share[warp][d] = x[k];
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int d = lane + 32 * k;
          if (d < R) {
            const bool second = g.t.interleaved ? d & 1 : d >= R / 2;
            const int pair = g.t.interleaved ? d >> 1 : second ? d - R / 2 : d;
            const float2 t = cos_sin(__ldg(g.t.turns + pair), pos);
            const float y = share[warp][g.t.interleaved ? d ^ 1 : second ? d - R / 2 : d + R / 2];
            x[k] = fmaf(x[k], t.x * g.t.amplitude, y * (second ? t.y : -t.y) * g.t.amplitude);
          }
        }
        __syncwarp();
      }
      if (m.part == 0) {
        bf16* out = static_cast<bf16*>(p.out) + m.token * p.ld_out + h * p.hs_out;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (lane + 32 * k < D) set_element(out + lane + 32 * k, x[k]);
        continue;
      }
      const int64_t row = row_at(at, g.c, h);
      if constexpr (MX) {
        uint8_t* codes = static_cast<uint8_t*>(m.part == 1 ? g.c.k : g.c.v) + row;
        uint8_t* units = (m.part == 1 ? g.c.k_scale : g.c.v_scale) + unit_at(at, g.c, h);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (32 * k >= D) break;
          float top = fabsf(x[k]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          const Unit u = unit_of(top);
          codes[lane + 32 * k] = static_cast<uint8_t>(codes2(x[k], 0.0f, u) & 0xFFu);
          if (lane == 0) units[k] = static_cast<uint8_t>(u.byte);
        }
      } else {
        bf16* out = static_cast<bf16*>(m.part == 1 ? g.c.k : g.c.v) + row;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (lane + 32 * k < D) set_element(out + lane + 32 * k, x[k]);
      }
    }
  }
}

template <bool I, int L>
cudaError_t launch_one(const Args& g, cudaStream_t s) {
  const bool partial = g.t.rot_dims < g.t.head_dim;  // (heads that turn in part have kernels of their own)
  auto* k = g.c.mx ? (partial ? kv_append_kernel<I, L, true, true> : kv_append_kernel<I, L, true, false>)
                   : (partial ? kv_append_kernel<I, L, false, true> : kv_append_kernel<I, L, false, false>);
  const int64_t ctas = (g.total + kWarps - 1) / kWarps, most = int64_t{1} << 30;  // (2^31 tokens have more than a grid's first dimension holds)
  return launch_pdl(k, dim3(static_cast<unsigned>(min(ctas, most)), static_cast<unsigned>((ctas + most - 1) / most)), dim3(kThreads), 0, s, g);
}

bool whole(const void* p, int64_t ld, int64_t hs, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * 2 % bytes == 0 && hs * 2 % bytes == 0;
}

}  // namespace

cudaError_t launch_kv_append(const Turn& f, const Heads (&part)[3], const Cache& c, const Batch& b, cudaStream_t stream) {
  Args g{};
  g.t = f;
  g.c = c;
  g.b = b;
  const int64_t bytes = f.interleaved ? 16 : 8;
  bool vec = f.head_dim % 8 == 0 && (f.interleaved || f.rot_dims % 8 == 0);
  int heads = 1;
  for (int p = 0; p < 3; ++p) {
    g.part[p] = part[p];
    heads = max(heads, part[p].n);
    if (part[p].n > 0) vec = vec && whole(part[p].in, part[p].ld_in, part[p].hs_in, p == 2 ? 8 : bytes) && (p != 0 || whole(part[p].out, part[p].ld_out, part[p].hs_out, bytes));
  }
  // runs of at least 8 heads, 64 items for each SM where there are as many
  const int64_t runs = min(static_cast<int64_t>((heads + 7) / 8), max(int64_t{1}, (int64_t{64} * num_sms() + f.tokens - 1) / f.tokens));
  g.per = static_cast<int>((heads + runs - 1) / runs);
  g.items = 0;
  for (int p = 0; p < 3; ++p) {
    g.first[p] = g.items;
    g.items += (part[p].n + g.per - 1) / g.per;
  }
  g.total = f.tokens * g.items;
  if (!vec) {
    const unsigned ctas = static_cast<unsigned>(min((g.total + kWarps - 1) / kWarps, int64_t{32} * num_sms()));
    return c.mx ? launch_pdl(kv_append_any_kernel<true>, dim3(ctas), dim3(kThreads), 0, stream, g) : launch_pdl(kv_append_any_kernel<false>, dim3(ctas), dim3(kThreads), 0, stream, g);
  }
  if (f.head_dim <= 64) return f.interleaved ? launch_one<true, 8>(g, stream) : launch_one<false, 8>(g, stream);
  if (f.head_dim <= 128) return f.interleaved ? launch_one<true, 16>(g, stream) : launch_one<false, 16>(g, stream);
  return f.interleaved ? launch_one<true, 32>(g, stream) : launch_one<false, 32>(g, stream);
}

}  // namespace fp8gb
