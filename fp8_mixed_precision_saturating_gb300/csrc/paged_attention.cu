// paged_attention.cu -- attention of new tokens over a paged cache.
//
// The simplest form: a warp per token and query head, one key after the other.
#include "heads.cuh"

namespace fp8gb {
namespace {

using namespace heads;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Args {
  Attention a;
  Cache c;
  Batch b;
};

template <int D, bool MX>
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(const __grid_constant__ Args g) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = i / g.a.q_heads;
  const int h = static_cast<int>(i - t * g.a.q_heads), hk = h / (g.a.q_heads / g.c.heads);
  if (t >= g.b.tokens) return;
  const Place at = place_of(t, g.b, lane);
  if (at.seq < 0) return;
  const bf16* q = static_cast<const bf16*>(g.a.q) + t * g.a.ld_q + h * g.a.hs_q;
  float x[E], o[E] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = element(q + lane * E + e);
  const int64_t capacity = static_cast<int64_t>(g.b.table_width) << g.c.page_bits;
  const int64_t end = min(min(at.pos + 1, capacity), static_cast<int64_t>(max(0, __ldg(g.b.kv_len + at.seq))));
  int64_t j = g.a.window > 0 ? max(int64_t{0}, at.pos + 1 - g.a.window) : 0;
  for (; j < end; ++j) {
    const int page = __ldg(g.b.page_table + at.seq * g.b.ld_table + (j >> g.c.page_bits));
    float k[E] = {}, v[E] = {};
    if (page >= 0 && page < g.c.pages) {
      const int slot = static_cast<int>(j & (g.c.page_size - 1));
      const int64_t row = page * g.c.page_stride + hk * g.c.head_stride + slot * g.c.token_stride + lane * E;
      if constexpr (MX) {
        const int64_t unit = ((static_cast<int64_t>(page) * g.c.heads + hk) * g.c.page_size + slot) * (D / 32) + lane * E / 32;
        auto get = [&](const void* codes, const uint8_t* units, float (&y)[E]) {
          const uint32_t u = units[unit];
          const float f = u == 0xFFu ? __int_as_float(0x7FFFFFFF) : exp2f(static_cast<float>(static_cast<int>(u) - 127));
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t b = static_cast<const uint8_t*>(codes)[row + e];
            const float w = __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7Fu) << 20)) * 0x1p120f;
            y[e] = w * f;
          }
        };
        get(g.c.k, g.c.k_scale, k);
        get(g.c.v, g.c.v_scale, v);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) k[e] = element(static_cast<const bf16*>(g.c.k) + row + e), v[e] = element(static_cast<const bf16*>(g.c.v) + row + e);
      }
    }
    float d = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) d = fmaf(x[e], k[e], d);
    d = row_sum<32>(d) * g.a.scale;
    const float n = fmaxf(m, d), base = n == -INFINITY ? 0.0f : n;
    const float old = __expf(m - base), w = __expf(d - base);
    l = l * old + w;
    m = n;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[e], o[e] * old);
  }
  bf16* out = static_cast<bf16*>(g.a.out) + t * g.a.ld_out + h * g.a.hs_out;
#pragma unroll
  for (int e = 0; e < E; ++e) set_element(out + lane * E + e, l == 0.0f ? 0.0f : o[e] / l);
  if (g.a.lse != nullptr && lane == 0) g.a.lse[t * g.a.q_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t paged_attention_workspace_bytes(const Attention&, const Cache&, const Batch&) { return 0; }

cudaError_t launch_paged_attention(const Attention& a, const Cache& c, const Batch& b, void*, cudaStream_t stream, const char**) {
  const Args g{a, c, b};
  const dim3 grid(static_cast<unsigned>((b.tokens * a.q_heads + kWarps - 1) / kWarps));
  if (c.head_dim == 64)
    return c.mx ? launch_pdl(paged_attention_kernel<64, true>, grid, dim3(kThreads), 0, stream, g) : launch_pdl(paged_attention_kernel<64, false>, grid, dim3(kThreads), 0, stream, g);
  return c.mx ? launch_pdl(paged_attention_kernel<128, true>, grid, dim3(kThreads), 0, stream, g) : launch_pdl(paged_attention_kernel<128, false>, grid, dim3(kThreads), 0, stream, g);
}

}  // namespace fp8gb
