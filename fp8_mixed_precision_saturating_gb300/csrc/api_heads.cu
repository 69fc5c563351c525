// api_heads.cu -- the C ABI of what stands between a block's projections (include/fp8gb.h): heads turned by their position, the paged
// cache and attention over it. Argument checks and the order of launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fp8gb.h"
#include "api.h"
#include "kernels.h"

using namespace fp8gb;

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1025;
constexpr int32_t kMaxHeads = 32767;

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }
fp8_status_t done(cudaError_t e, const char* who) { return e == cudaSuccess ? FP8_OK : cuda_fail(e, who); }

#define FP8GB_TRY(call)            \
  do {                             \
    const fp8_status_t st_ = (call); \
    if (st_ != FP8_OK) return st_; \
  } while (0)

// Two nested strides whose rows of `dim` elements do not overlap: n0 at s0 within the step s1 of n1, or the other way round.
bool nested(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t dim) {
  using wide = __int128;
  const bool inner = n0 <= 1 || s0 >= dim, outer = n1 <= 1 || static_cast<wide>(s1) >= static_cast<wide>(n0 - 1) * (n0 > 1 ? s0 : 0) + dim;
  return inner && outer;
}

// A head tensor [tokens, heads, dim].
fp8_status_t check_heads(const void* p, int64_t ld, int64_t hs, int64_t tokens, int64_t heads, int64_t dim, int64_t size, const char* who, const char* name) {
  if (p == nullptr || tokens == 0 || heads == 0) return FP8_OK;
  if (!nested(heads, hs, tokens, ld, dim) && !nested(tokens, ld, heads, hs, dim))
    return fail(FP8_ERR_INVALID_ARG, "%s: rows of %s overlap (ld %lld, head stride %lld)", who, name, (long long)ld, (long long)hs);
  if (!aligned_to(p, size)) return fail(FP8_ERR_ALIGNMENT, "%s: %s is not aligned to its elements", who, name);
  return FP8_OK;
}

// The same rows in the same places, if the same address.
fp8_status_t check_in_place(const void* x, int64_t ld_x, int64_t hs_x, const void* y, int64_t ld_y, int64_t hs_y, int64_t tokens, int64_t heads, const char* who, const char* name) {
  if (x == nullptr || x != y || (tokens <= 1 && heads <= 1)) return FP8_OK;
  if ((tokens > 1 && ld_x != ld_y) || (heads > 1 && hs_x != hs_y)) return fail(FP8_ERR_INVALID_ARG, "%s: %s in place with other strides", who, name);
  return FP8_OK;
}

fp8_status_t check_turn(const fp8_qk_rope_t* f, const char* who) {
  if (f == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null arguments", who);
  if (f->tokens < 0 || f->q_heads < 0 || f->k_heads < 0 || f->head_dim < 1) return fail(FP8_ERR_INVALID_ARG, "%s: negative size, or no head_dim", who);
  if (f->dt != FP8_DT_BF16 && f->dt != FP8_DT_F32) return fail(FP8_ERR_INVALID_ARG, "%s: unknown type", who);
  if (f->layout != FP8_ROPE_HALF && f->layout != FP8_ROPE_INTERLEAVED) return fail(FP8_ERR_INVALID_ARG, "%s: unknown layout", who);
  if (f->norm < FP8_NORM_NONE || f->norm > FP8_NORM_LAYER) return fail(FP8_ERR_INVALID_ARG, "%s: unknown norm", who);
  if (f->rot_dims < 0 || f->rot_dims % 2 != 0 || f->rot_dims > f->head_dim)
    return fail(FP8_ERR_INVALID_ARG, "%s: rot_dims must be even, 0 .. head_dim", who);
  if (!(f->eps >= 0.0f) || !std::isfinite(f->eps)) return fail(FP8_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (!std::isfinite(f->amplitude) || f->amplitude == 0.0f) return fail(FP8_ERR_INVALID_ARG, "%s: amplitude must be finite and not 0", who);
  if (f->rot_dims > 0 && f->turns == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null turns", who);
  if (f->norm == FP8_NORM_NONE && (f->w_q != nullptr || f->w_k != nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: w_q or w_k without a norm", who);
  if (f->norm == FP8_NORM_LAYER) return fail(FP8_ERR_UNSUPPORTED, "%s: heads have no layer norm here", who);
  if (f->tokens > kMaxDim || f->q_heads > kMaxHeads || f->k_heads > kMaxHeads) return fail(FP8_ERR_UNSUPPORTED, "%s: 2^31 - 1024 tokens or 32768 heads or more", who);
  if (f->head_dim > 256) return fail(FP8_ERR_UNSUPPORTED, "%s: head_dim above 256", who);
  if (!aligned_to(f->turns, 8) || !aligned_to(f->pos, 4) || !aligned_to(f->w_q, 4) || !aligned_to(f->w_k, 4))
    return fail(FP8_ERR_ALIGNMENT, "%s: turns, pos or a weight is not aligned to its elements", who);
  const int64_t size = f->dt == FP8_DT_F32 ? 4 : 2;
  FP8GB_TRY(check_heads(f->q, f->ld_q, f->hs_q, f->tokens, f->q_heads, f->head_dim, size, who, "q"));
  FP8GB_TRY(check_heads(f->k, f->ld_k, f->hs_k, f->tokens, f->k_heads, f->head_dim, size, who, "k"));
  FP8GB_TRY(check_heads(f->q_out, f->ld_q_out, f->hs_q_out, f->tokens, f->q_heads, f->head_dim, size, who, "q_out"));
  FP8GB_TRY(check_heads(f->k_out, f->ld_k_out, f->hs_k_out, f->tokens, f->k_heads, f->head_dim, size, who, "k_out"));
  FP8GB_TRY(check_in_place(f->q, f->ld_q, f->hs_q, f->q_out, f->ld_q_out, f->hs_q_out, f->tokens, f->q_heads, who, "q"));
  return check_in_place(f->k, f->ld_k, f->hs_k, f->k_out, f->ld_k_out, f->hs_k_out, f->tokens, f->k_heads, who, "k");
}

Turn to_turn(const fp8_qk_rope_t* f) {
  return Turn{f->tokens, f->head_dim, f->rot_dims, f->dt == FP8_DT_F32, f->layout == FP8_ROPE_INTERLEAVED, f->norm == FP8_NORM_RMS, f->eps, f->amplitude, f->turns, f->pos};
}
Heads q_of(const fp8_qk_rope_t* f) { return Heads{f->q, f->q_out, f->ld_q, f->hs_q, f->ld_q_out, f->hs_q_out, f->w_q, f->q_heads}; }
Heads k_of(const fp8_qk_rope_t* f) { return Heads{f->k, f->k_out, f->ld_k, f->hs_k, f->ld_k_out, f->hs_k_out, f->w_k, f->k_heads}; }

fp8_status_t check_grad(const fp8_qk_rope_t* f, const fp8_qk_rope_grad_t* b, const char* who) {
  FP8GB_TRY(check_turn(f, who));
  if (b == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null gradients", who);
  if (f->norm == FP8_NORM_NONE && (b->dw_q != nullptr || b->dw_k != nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: dw_q or dw_k without a norm", who);
  const int64_t size = f->dt == FP8_DT_F32 ? 4 : 2;
  FP8GB_TRY(check_heads(b->dq_out, b->ld_dq_out, b->hs_dq_out, f->tokens, f->q_heads, f->head_dim, size, who, "dq_out"));
  FP8GB_TRY(check_heads(b->dk_out, b->ld_dk_out, b->hs_dk_out, f->tokens, f->k_heads, f->head_dim, size, who, "dk_out"));
  FP8GB_TRY(check_heads(b->dq, b->ld_dq, b->hs_dq, f->tokens, f->q_heads, f->head_dim, size, who, "dq"));
  FP8GB_TRY(check_heads(b->dk, b->ld_dk, b->hs_dk, f->tokens, f->k_heads, f->head_dim, size, who, "dk"));
  FP8GB_TRY(check_in_place(b->dq_out, b->ld_dq_out, b->hs_dq_out, b->dq, b->ld_dq, b->hs_dq, f->tokens, f->q_heads, who, "dq"));
  FP8GB_TRY(check_in_place(b->dk_out, b->ld_dk_out, b->hs_dk_out, b->dk, b->ld_dk, b->hs_dk, f->tokens, f->k_heads, who, "dk"));
  if (!aligned_to(b->dw_q, 4) || !aligned_to(b->dw_k, 4)) return fail(FP8_ERR_ALIGNMENT, "%s: dw_q or dw_k is not aligned to its elements", who);
  return FP8_OK;
}

fp8_status_t check_cache(const fp8_kv_cache_t* c, const char* who) {
  if (c == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null cache", who);
  if (c->format != FP8_KV_BF16 && c->format != FP8_KV_MX_E4M3) return fail(FP8_ERR_INVALID_ARG, "%s: unknown cache format %d", who, (int)c->format);
  if (c->pages < 0 || c->heads < 1 || c->head_dim < 1 || c->page_size < 1) return fail(FP8_ERR_INVALID_ARG, "%s: negative or no size of the cache", who);
  const bool mx = c->format == FP8_KV_MX_E4M3;
  if (c->page_size < 8 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(FP8_ERR_UNSUPPORTED, "%s: page_size must be a power of two, 8 .. 4096", who);
  if (c->heads > kMaxHeads || c->head_dim > 256) return fail(FP8_ERR_UNSUPPORTED, "%s: cache of 32768 heads or more, or head_dim above 256", who);
  if (mx && c->head_dim % 32 != 0) return fail(FP8_ERR_UNSUPPORTED, "%s: an 8-bit cache needs head_dim %% 32 == 0", who);
  if (c->pages > 0 && (c->k == nullptr || c->v == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: null cache buffers", who);
  if (mx && c->pages > 0 && (c->k_scale == nullptr || c->v_scale == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: an 8-bit cache needs its scales", who);
  if (!mx && (c->k_scale != nullptr || c->v_scale != nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: a bf16 cache has no scales", who);
  const int64_t P = c->page_size, H = c->heads, D = c->head_dim, ts = c->token_stride, hs = c->head_stride, ps = c->page_stride;
  const bool tokens_inside = nested(P, ts, H, hs, D), heads_inside = nested(H, hs, P, ts, D);
  const int64_t limit = 1ll << 40;
  if (ts > limit || hs > limit || ps > limit) return fail(FP8_ERR_UNSUPPORTED, "%s: a stride of the cache above 2^40", who);
  const int64_t span = (P - 1) * ts + (H > 1 ? (H - 1) * hs : 0) + D;
  if ((!tokens_inside && !heads_inside) || (c->pages > 1 && ps < span)) return fail(FP8_ERR_INVALID_ARG, "%s: rows of the cache overlap", who);
  const int64_t unit = mx ? 16 : 8;  // elements of 16 bytes
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) || ts % unit != 0 || (H > 1 && hs % unit != 0) || (c->pages > 1 && ps % unit != 0))
    return fail(FP8_ERR_ALIGNMENT, "%s: the cache's buffers and strides must be of whole 16 bytes", who);
  return FP8_OK;
}

fp8_status_t check_batch(const fp8_kv_batch_t* b, const char* who) {
  if (b == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null batch", who);
  if (b->tokens < 0 || b->seqs < 0 || b->table_width < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size of the batch", who);
  if (b->tokens > kMaxDim || b->seqs > kMaxDim) return fail(FP8_ERR_UNSUPPORTED, "%s: 2^31 - 1024 tokens or sequences, or more", who);
  if (b->seqs > 0 && b->tokens > 0 && (b->q_start == nullptr || b->kv_len == nullptr || (b->page_table == nullptr && b->table_width > 0)))
    return fail(FP8_ERR_INVALID_ARG, "%s: null q_start, kv_len or page_table", who);
  if (b->seqs > 1 && b->ld_table < b->table_width) return fail(FP8_ERR_INVALID_ARG, "%s: ld_table (%lld) < table_width (%d)", who, (long long)b->ld_table, (int)b->table_width);
  if (!aligned_to(b->q_start, 4) || !aligned_to(b->kv_len, 4) || !aligned_to(b->page_table, 4))
    return fail(FP8_ERR_ALIGNMENT, "%s: q_start, kv_len or page_table is not aligned to its elements", who);
  return FP8_OK;
}

Cache to_cache(const fp8_kv_cache_t* c) {
  int bits = 0;
  while ((1 << bits) < c->page_size) ++bits;
  return Cache{c->k, c->v, c->k_scale, c->v_scale, c->format == FP8_KV_MX_E4M3, c->pages, c->page_size, bits, c->heads, c->head_dim, c->page_stride, c->head_stride, c->token_stride};
}
Batch to_batch(const fp8_kv_batch_t* b) { return Batch{b->tokens, b->ld_table, b->seqs, b->table_width, b->q_start, b->kv_len, b->page_table}; }

Attention to_attention(const fp8_paged_attention_t* a) { return Attention{a->q_heads, a->window, a->scale, a->q, a->out, a->ld_q, a->hs_q, a->ld_out, a->hs_out, a->lse}; }

fp8_status_t check_attention(const fp8_paged_attention_t* a, const fp8_kv_cache_t* c, const fp8_kv_batch_t* b, const char* who) {
  if (a == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null arguments", who);
  FP8GB_TRY(check_cache(c, who));
  FP8GB_TRY(check_batch(b, who));
  if (a->q_heads < 1 || a->window < 0) return fail(FP8_ERR_INVALID_ARG, "%s: no query heads, or a negative window", who);
  if (!std::isfinite(a->scale)) return fail(FP8_ERR_INVALID_ARG, "%s: scale must be finite", who);
  if (a->q_heads % c->heads != 0) return fail(FP8_ERR_INVALID_ARG, "%s: q_heads (%d) is no multiple of the cache's heads (%d)", who, (int)a->q_heads, (int)c->heads);
  if (c->head_dim != 64 && c->head_dim != 128) return fail(FP8_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", who);
  if (a->q_heads / c->heads > 128) return fail(FP8_ERR_UNSUPPORTED, "%s: more than 128 query heads for one of the cache's", who);
  if (b->seqs > kAttendMaxSeqs) return fail(FP8_ERR_UNSUPPORTED, "%s: more than %d sequences", who, kAttendMaxSeqs);
  if (a->q_heads > kMaxHeads) return fail(FP8_ERR_UNSUPPORTED, "%s: 32768 heads or more", who);
  if (b->tokens > 0 && (a->q == nullptr || a->out == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: null q or out", who);
  FP8GB_TRY(check_heads(a->q, a->ld_q, a->hs_q, b->tokens, a->q_heads, c->head_dim, 2, who, "q"));
  FP8GB_TRY(check_heads(a->out, a->ld_out, a->hs_out, b->tokens, a->q_heads, c->head_dim, 2, who, "out"));
  FP8GB_TRY(check_in_place(a->q, a->ld_q, a->hs_q, a->out, a->ld_out, a->hs_out, b->tokens, a->q_heads, who, "q"));
  const int64_t limit = 1ll << 40;
  if (a->ld_q > limit || a->hs_q > limit) return fail(FP8_ERR_UNSUPPORTED, "%s: a stride of q above 2^40", who);
  auto whole = [&](int64_t ld, int64_t hs) { return (b->tokens <= 1 || ld % 8 == 0) && (a->q_heads <= 1 || hs % 8 == 0); };
  if (!aligned16(a->q) || !aligned16(a->out) || !whole(a->ld_q, a->hs_q) || !whole(a->ld_out, a->hs_out))
    return fail(FP8_ERR_ALIGNMENT, "%s: q and out must be 16-byte aligned with strides of multiples of 8", who);
  if (!aligned_to(a->lse, 4)) return fail(FP8_ERR_ALIGNMENT, "%s: lse is not aligned to its elements", who);
  const char* why = paged_attention_refusal(to_attention(a), to_cache(c), to_batch(b));
  if (why != nullptr) return fail(FP8_ERR_UNSUPPORTED, "%s: %s", who, why);
  return FP8_OK;
}

}  // namespace

extern "C" {

fp8_status_t fp8_rope_turns(int32_t rot_dims, double base, fp8_rope_scaling_t kind, double factor, double original, double low, double high, uint64_t* turns) {
  const char* who = "fp8_rope_turns";
  if (rot_dims < 0 || rot_dims % 2 != 0) return fail(FP8_ERR_INVALID_ARG, "%s: rot_dims must be even and >= 0", who);
  if (rot_dims > 256) return fail(FP8_ERR_UNSUPPORTED, "%s: rot_dims above 256", who);
  if (kind < FP8_ROPE_PLAIN || kind > FP8_ROPE_PARTS_BY_INDEX) return fail(FP8_ERR_INVALID_ARG, "%s: unknown scaling %d", who, (int)kind);
  if (!std::isfinite(base) || !(base > 1.0)) return fail(FP8_ERR_INVALID_ARG, "%s: base must be finite and above 1", who);
  const bool parts = kind == FP8_ROPE_PARTS || kind == FP8_ROPE_PARTS_BY_INDEX;
  if (kind != FP8_ROPE_PLAIN && !(std::isfinite(factor) && factor > 0.0)) return fail(FP8_ERR_INVALID_ARG, "%s: factor must be finite and above 0", who);
  if (kind == FP8_ROPE_BASE && rot_dims < 4) return fail(FP8_ERR_INVALID_ARG, "%s: a stretched base needs rot_dims >= 4", who);
  if (parts && !(std::isfinite(original) && original > 0.0 && std::isfinite(high) && low > 0.0 && low < high))
    return fail(FP8_ERR_INVALID_ARG, "%s: the parts need original > 0 and 0 < low < high", who);
  if (rot_dims > 0 && turns == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null turns", who);
  const double two_pi = 6.283185307179586476925;
  if (kind == FP8_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot_dims) / (rot_dims - 2));
  // the (real) index of a frequency that turns r times over the original length
  auto index_of = [&](double r) { return 0.5 * rot_dims * std::log(original / (two_pi * r)) / std::log(base); };
  for (int i = 0; i < rot_dims / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dims) / two_pi;  // turns per position
    double s = kind == FP8_ROPE_LINEAR ? 0.0 : 1.0;
    if (kind == FP8_ROPE_PARTS) s = (original * f - low) / (high - low);
    if (kind == FP8_ROPE_PARTS_BY_INDEX) s = (index_of(low) - i) / (index_of(low) - index_of(high));
    s = std::fmin(std::fmax(s, 0.0), 1.0);
    if (s < 1.0) f = s * f + (1.0 - s) * (f / factor);
    f -= std::floor(f);
    const double scaled = std::nearbyint(f * 18446744073709551616.0);
    turns[i] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
  }
  return FP8_OK;
}

fp8_status_t fp8_qk_rope_fwd(const fp8_qk_rope_t* f, void* stream) {
  const char* who = "fp8_qk_rope_fwd";
  FP8GB_TRY(check_turn(f, who));
  Heads part[2] = {q_of(f), k_of(f)};
  bool any = false;
  for (Heads& p : part) {
    if ((p.in == nullptr) != (p.out == nullptr) && p.n > 0 && f->tokens > 0)
      return fail(FP8_ERR_INVALID_ARG, "%s: %s without %s_out, or the other way round", who, &p == part ? "q" : "k", &p == part ? "q" : "k");
    if (p.in == nullptr) p.n = 0;
    any = any || p.n > 0;
  }
  if (f->tokens > 0 && !any) return fail(FP8_ERR_INVALID_ARG, "%s: no output", who);
  if (f->tokens == 0) return FP8_OK;
  return done(launch_qk_rope_fwd(to_turn(f), part, static_cast<cudaStream_t>(stream)), who);
}

int64_t fp8_qk_rope_bwd_workspace_bytes(const fp8_qk_rope_t* f, const fp8_qk_rope_grad_t* b) {
  const char* who = "fp8_qk_rope_bwd_workspace_bytes";
  if (check_grad(f, b, who) != FP8_OK) return -1;
  return b->dw_q == nullptr && b->dw_k == nullptr ? 0 : qk_rope_bwd_workspace_bytes(to_turn(f));
}

fp8_status_t fp8_qk_rope_bwd(const fp8_qk_rope_t* f, const fp8_qk_rope_grad_t* b, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "fp8_qk_rope_bwd";
  FP8GB_TRY(check_grad(f, b, who));
  Heads part[2] = {q_of(f), k_of(f)};
  TurnGrad grad[2] = {{b->dq_out, b->dq, b->ld_dq_out, b->hs_dq_out, b->ld_dq, b->hs_dq, b->dw_q}, {b->dk_out, b->dk, b->ld_dk_out, b->hs_dk_out, b->ld_dk, b->hs_dk, b->dw_k}};
  bool any = false;
  for (int p = 0; p < 2; ++p) {
    const char* name = p == 0 ? "q" : "k";
    const bool some = f->tokens > 0 && part[p].n > 0;
    if (some && grad[p].dy == nullptr && (grad[p].dx != nullptr || grad[p].dw != nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: d%s or dw_%s without d%s_out", who, name, name, name);
    if (some && grad[p].dy != nullptr && f->norm != FP8_NORM_NONE && part[p].in == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: the norm's gradient needs %s", who, name);
    if (grad[p].dy == nullptr || (grad[p].dx == nullptr && grad[p].dw == nullptr)) part[p].n = 0;
    any = any || part[p].n > 0;
  }
  if (workspace_bytes < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative workspace size", who);
  if (!aligned16(workspace)) return fail(FP8_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", who);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (f->tokens == 0 || !any) {  // sums over nothing
    for (const TurnGrad& g : grad)
      if (g.dw != nullptr) FP8GB_TRY(done(cudaMemsetAsync(g.dw, 0, f->head_dim * 4, s), who));
    return f->tokens > 0 && (f->q_heads > 0 || f->k_heads > 0) && b->dw_q == nullptr && b->dw_k == nullptr ? fail(FP8_ERR_INVALID_ARG, "%s: no output", who) : FP8_OK;
  }
  const int64_t need = b->dw_q == nullptr && b->dw_k == nullptr ? 0 : qk_rope_bwd_workspace_bytes(to_turn(f));
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(FP8_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who, (long long)(workspace ? workspace_bytes : 0), (long long)need);
  return done(launch_qk_rope_bwd(to_turn(f), part, grad, workspace, s), who);
}

fp8_status_t fp8_kv_append(const fp8_qk_rope_t* f, const fp8_kv_cache_t* c, const fp8_kv_batch_t* b, void* stream) {
  const char* who = "fp8_kv_append";
  FP8GB_TRY(check_turn(f, who));
  FP8GB_TRY(check_cache(c, who));
  FP8GB_TRY(check_batch(b, who));
  if (f->dt != FP8_DT_BF16) return fail(FP8_ERR_UNSUPPORTED, "%s: the head tensors must be bf16", who);
  if (f->k_heads != c->heads || f->head_dim != c->head_dim)
    return fail(FP8_ERR_INVALID_ARG, "%s: %d heads of %d into a cache of %d of %d", who, (int)f->k_heads, (int)f->head_dim, (int)c->heads, (int)c->head_dim);
  if (f->tokens != b->tokens) return fail(FP8_ERR_INVALID_ARG, "%s: %lld tokens, and %lld in the batch", who, (long long)f->tokens, (long long)b->tokens);
  if (f->k_out != nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: the keys go into the cache, not to k_out", who);
  FP8GB_TRY(check_heads(f->v, f->ld_v, f->hs_v, f->tokens, f->k_heads, f->head_dim, 2, who, "v"));
  if (f->tokens > 0 && (f->k == nullptr || f->v == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: null k or v", who);
  if (f->tokens > 0 && f->q_heads > 0 && (f->q == nullptr) != (f->q_out == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: q without q_out, or the other way round", who);
  if (f->tokens == 0 || b->seqs == 0) return FP8_OK;
  Heads part[3] = {q_of(f), k_of(f), Heads{f->v, nullptr, f->ld_v, f->hs_v, 0, 0, nullptr, f->k_heads}};
  if (f->q == nullptr) part[0].n = 0;
  return done(launch_kv_append(to_turn(f), part, to_cache(c), to_batch(b), static_cast<cudaStream_t>(stream)), who);
}

int64_t fp8_paged_attention_workspace_bytes(const fp8_paged_attention_t* a, const fp8_kv_cache_t* c, const fp8_kv_batch_t* b) {
  if (check_attention(a, c, b, "fp8_paged_attention_workspace_bytes") != FP8_OK) return -1;
  return paged_attention_workspace_bytes(to_attention(a), to_cache(c), to_batch(b));
}

fp8_status_t fp8_paged_attention(const fp8_paged_attention_t* a, const fp8_kv_cache_t* c, const fp8_kv_batch_t* b, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
  const char* who = "fp8_paged_attention";
  FP8GB_TRY(check_attention(a, c, b, who));
  if (workspace_bytes < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative workspace size", who);
  if (!aligned16(workspace)) return fail(FP8_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", who);
  if (b->tokens == 0 || b->seqs == 0) return FP8_OK;
  const Attention at = to_attention(a);
  const Cache cache = to_cache(c);
  const Batch batch = to_batch(b);
  const int64_t need = paged_attention_workspace_bytes(at, cache, batch);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(FP8_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who, (long long)(workspace ? workspace_bytes : 0), (long long)need);
  const char* why = nullptr;
  const cudaError_t e = launch_paged_attention(at, cache, batch, workspace, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess && why != nullptr) return fail(FP8_ERR_CUDA, "%s: %s", who, why);
  return done(e, who);
}

}  // extern "C"
