// api4.cu -- the C ABI of the 4-bit operands and of the norms around a block (include/fp8gb.h):
// argument checks and the order of launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fp8gb.h"
#include "api.h"
#include "fp4.cuh"
#include "kernels.h"

using namespace fp8gb;

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1025;  // the end of a tile that a dimension ends in is still a 32-bit number

bool known(fp4_format_t f) { return f == FP4_NVFP4 || f == FP4_MXFP4; }
bool known(fp8_dtype_t t) { return t == FP8_DT_BF16 || t == FP8_DT_F32; }
bool known_norm(int32_t k) { return k >= FP8_NORM_NONE && k <= FP8_NORM_LAYER; }
bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

fp8_status_t check_device(const char* who) {
  int d = 0;
  const cudaError_t e = cudaGetDevice(&d);
  return e == cudaSuccess ? FP8_OK : cuda_fail(e, who);
}

fp8_status_t done(cudaError_t e, const char* who) { return e == cudaSuccess ? FP8_OK : cuda_fail(e, who); }

// A matrix argument of the norms: [tokens, width] of `size`-byte elements.
fp8_status_t check_matrix(const void* p, int64_t ld, int64_t rows, int64_t width, int64_t size, const char* who, const char* name) {
  if (p == nullptr || rows == 0) return FP8_OK;
  if (ld < width && rows > 1) return fail(FP8_ERR_INVALID_ARG, "%s: ld of %s (%lld) < width (%lld)", who, name, (long long)ld, (long long)width);
  if (!aligned_to(p, size)) return fail(FP8_ERR_ALIGNMENT, "%s: %s is not aligned to its elements", who, name);
  return FP8_OK;
}

fp8_status_t check_vector(const void* p, const char* who, const char* name) {
  return aligned_to(p, 4) ? FP8_OK : fail(FP8_ERR_ALIGNMENT, "%s: %s is not aligned to its elements", who, name);
}

#define FP8GB_TRY(call)                       \
  do {                                        \
    const fp8_status_t st_ = (call);          \
    if (st_ != FP8_OK) return st_;            \
  } while (0)

// What forward and backward ask of the shared arguments.
fp8_status_t check_norm(const fp8_block_norm_t* f, const char* who) {
  if (f == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null arguments", who);
  if (f->tokens < 0 || f->width < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", who);
  if (!known(static_cast<fp8_dtype_t>(f->stream_dt)) || !known(static_cast<fp8_dtype_t>(f->block_dt)))
    return fail(FP8_ERR_INVALID_ARG, "%s: unknown type", who);
  if (!known_norm(f->post) || !known_norm(f->pre)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown norm", who);
  if (!(f->eps >= 0.0f) || !std::isfinite(f->eps)) return fail(FP8_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (f->tokens > kMaxDim || f->width > kMaxDim) return fail(FP8_ERR_UNSUPPORTED, "%s: dimension >= 2^31 - 1024", who);
  if (f->gate != nullptr && f->gate_rows <= 0) return fail(FP8_ERR_INVALID_ARG, "%s: a gate needs gate_rows > 0", who);
  if (f->post == FP8_NORM_NONE && (f->w_post != nullptr || f->b_post != nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: w_post or b_post without a norm after the block", who);
  if (f->pre == FP8_NORM_NONE && (f->w_pre != nullptr || f->b_pre != nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: w_pre or b_pre without a norm before the next block", who);
  if (f->tokens > 0 && f->width > 0 && f->o == nullptr && (f->post != FP8_NORM_NONE || f->gate != nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: a norm after the block or a gate without o", who);
  const int64_t ss = f->stream_dt == FP8_DT_F32 ? 4 : 2, bs = f->block_dt == FP8_DT_F32 ? 4 : 2;
  const int64_t groups = f->gate != nullptr && f->tokens > 0 ? (f->tokens - 1) / f->gate_rows + 1 : 0;
  FP8GB_TRY(check_matrix(f->r, f->ld_r, f->tokens, f->width, ss, who, "r"));
  FP8GB_TRY(check_matrix(f->o, f->ld_o, f->tokens, f->width, bs, who, "o"));
  FP8GB_TRY(check_matrix(f->gate, f->ld_gate, groups, f->width, bs, who, "gate"));
  FP8GB_TRY(check_matrix(f->r_out, f->ld_r_out, f->tokens, f->width, ss, who, "r_out"));
  const void* vec[] = {f->res_scale, f->w_post, f->b_post, f->w_pre, f->b_pre};
  for (const void* v : vec) FP8GB_TRY(check_vector(v, who, "a parameter"));
  if (!aligned_to(f->stat_post, 8) || !aligned_to(f->stat_pre, 8))
    return fail(FP8_ERR_ALIGNMENT, "%s: the statistics must be 8-byte aligned", who);
  return FP8_OK;
}

NormFwd to_fwd(const fp8_block_norm_t* f) {
  NormFwd n{};
  n.tokens = f->tokens;
  n.width = f->width;
  n.stream_f32 = f->stream_dt == FP8_DT_F32;
  n.block_f32 = f->block_dt == FP8_DT_F32;
  n.post = f->post;
  n.pre = f->pre;
  n.eps = f->eps;
  n.r = f->r;
  n.o = f->o;
  n.gate = f->gate;
  n.ld_r = f->ld_r;
  n.ld_o = f->ld_o;
  n.ld_gate = f->ld_gate;
  // a gate of more rows than there are tokens is one for all of them; past here its ends and counts fit 64 bits
  n.gate_rows = f->gate != nullptr && f->gate_rows < f->tokens ? f->gate_rows : f->tokens;
  n.res_scale = f->res_scale;
  n.w_post = f->w_post;
  n.b_post = f->b_post;
  n.w_pre = f->w_pre;
  n.b_pre = f->b_pre;
  n.r_out = f->r_out;
  n.h = f->h;
  n.ld_r_out = f->ld_r_out;
  n.ld_h = f->ld_h;
  n.hq = static_cast<uint8_t*>(f->hq);
  n.hsf = static_cast<uint8_t*>(f->hsf);
  n.h_fmt = f->h_fmt;
  n.h_scale = f->h_scale;
  n.stat_post = f->stat_post;
  n.stat_pre = f->stat_pre;
  return n;
}

}  // namespace

extern "C" {

int64_t fp4_row_bytes(int64_t K) { return K < 0 ? -1 : fp4::row_bytes(K); }

int64_t fp4_scale_bytes(fp4_format_t fmt, int64_t MN, int64_t K) {
  if (!known(fmt) || MN < 0 || K < 0) return -1;
  return (MN + 127) / 128 * fp4::atoms_along(fmt, K) * 512;
}

fp8_status_t fp4_quantize(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld, fp4_format_t fmt,
                          fp8_scaling_t mode, const fp8_tensor_state_t* st, void* q, void* sf, void* qT, void* sfT,
                          void* stream) {
  const char* who = "fp4_quantize";
  if (rows < 0 || cols < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", who);
  if (!known(fmt)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format %d", who, (int)fmt);
  if (mode != FP8_SCALE_CURRENT && mode != FP8_SCALE_DELAYED)
    return fail(FP8_ERR_INVALID_ARG, "%s: unknown scaling mode %d", who, (int)mode);
  if ((q == nullptr) != (sf == nullptr) || (qT == nullptr) != (sfT == nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: codes and their scales go together", who);
  const bool empty = rows == 0 || cols == 0;
  if (!empty && q == nullptr && qT == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: no output", who);
  if (!empty && x_bf16 == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null input", who);
  if (ld < cols) return fail(FP8_ERR_INVALID_ARG, "%s: ld (%lld) < cols (%lld)", who, (long long)ld, (long long)cols);
  if (st != nullptr && fmt != FP4_NVFP4) return fail(FP8_ERR_INVALID_ARG, "%s: MXFP4 has no tensor scale", who);
  if (st == nullptr && mode == FP8_SCALE_DELAYED)
    return fail(FP8_ERR_INVALID_ARG, "%s: delayed scaling needs a state", who);
  if (st != nullptr) FP8GB_TRY(check_state(st, mode, who));
  if (rows > kMaxDim || cols > kMaxDim) return fail(FP8_ERR_UNSUPPORTED, "%s: dimension >= 2^31 - 1024", who);
  if (!aligned16(q) || !aligned16(sf) || !aligned16(qT) || !aligned16(sfT))
    return fail(FP8_ERR_ALIGNMENT, "%s: the codes and scales must be 16-byte aligned", who);
  if (!aligned_to(x_bf16, 2)) return fail(FP8_ERR_ALIGNMENT, "%s: x is not aligned to its elements", who);
  if (empty) return FP8_OK;
  return done(launch_quant4(fmt, mode == FP8_SCALE_DELAYED, x_bf16, rows, cols, ld, to_qs(st), q, sf, qT, sfT,
                            static_cast<cudaStream_t>(stream)),
              who);
}

fp8_status_t fp4_dequantize(const void* q, const void* sf, int64_t MN, int64_t K, fp4_format_t fmt,
                            const float* scale_inv, void* y, fp8_dtype_t dt, int64_t ldy, void* stream) {
  const char* who = "fp4_dequantize";
  if (MN < 0 || K < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", who);
  if (!known(fmt)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format %d", who, (int)fmt);
  if (!known(dt)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown type %d", who, (int)dt);
  if (ldy < K) return fail(FP8_ERR_INVALID_ARG, "%s: ldy (%lld) < K (%lld)", who, (long long)ldy, (long long)K);
  const bool empty = MN == 0 || K == 0;
  if (!empty && (q == nullptr || sf == nullptr || y == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: null codes, scales or output", who);
  if (MN > kMaxDim || K > kMaxDim) return fail(FP8_ERR_UNSUPPORTED, "%s: dimension >= 2^31 - 1024", who);
  if (!aligned16(q) || !aligned16(sf)) return fail(FP8_ERR_ALIGNMENT, "%s: the codes and scales must be 16-byte aligned", who);
  if (!aligned_to(y, dt == FP8_DT_F32 ? 4 : 2) || !aligned_to(scale_inv, 4))
    return fail(FP8_ERR_ALIGNMENT, "%s: y or scale_inv is not aligned to its elements", who);
  if (empty) return FP8_OK;
  return done(launch_dequant4(fmt, dt == FP8_DT_F32, q, sf, MN, K, scale_inv, y, ldy, static_cast<cudaStream_t>(stream)), who);
}

fp8_status_t fp4_scaled_mm(const void* A, const void* sfa, const void* B, const void* sfb, int64_t M, int64_t N, int64_t K,
                           fp4_format_t fmt, const float* scale_inv_a, const float* scale_inv_b, void* C, fp8_dtype_t dt,
                           int64_t ldc, void* stream) {
  const char* who = "fp4_scaled_mm";
  if (M < 0 || N < 0 || K < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", who);
  if (!known(fmt)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format %d", who, (int)fmt);
  if (!known(dt)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown type %d", who, (int)dt);
  if (ldc < N) return fail(FP8_ERR_INVALID_ARG, "%s: ldc (%lld) < N (%lld)", who, (long long)ldc, (long long)N);
  const bool empty = M == 0 || N == 0;
  if (!empty && C == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null C", who);
  if (!empty && K > 0 && (A == nullptr || B == nullptr || sfa == nullptr || sfb == nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: null A, B or scales", who);
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return fail(FP8_ERR_UNSUPPORTED, "%s: dimension >= 2^31 - 1024", who);
  if (!aligned16(A) || !aligned16(B) || !aligned16(sfa) || !aligned16(sfb) || !aligned16(C))
    return fail(FP8_ERR_ALIGNMENT, "%s: A, B, their scales and C must be 16-byte aligned", who);
  if (ldc % (dt == FP8_DT_F32 ? 4 : 8) != 0)
    return fail(FP8_ERR_ALIGNMENT, "%s: ldc must be a multiple of %d", who, dt == FP8_DT_F32 ? 4 : 8);
  if (!aligned_to(scale_inv_a, 4) || !aligned_to(scale_inv_b, 4))
    return fail(FP8_ERR_ALIGNMENT, "%s: scale_inv_a or scale_inv_b is not aligned to its elements", who);
  if (empty) return FP8_OK;
  const int64_t size = dt == FP8_DT_F32 ? 4 : 2;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return done(cudaMemset2DAsync(C, ldc * size, 0, N * size, M, s), who);
  const Mm4Args g{A, sfa, B, sfb, M, N, K, (int)fmt, scale_inv_a, scale_inv_b, C, dt == FP8_DT_F32, ldc};
  const char* why = nullptr;
  const cudaError_t e = launch_mm4(g, s, &why);
  if (e != cudaSuccess && why != nullptr) return fail(FP8_ERR_CUDA, "%s: %s", who, why);
  return done(e, who);
}

fp8_status_t fp8_block_norm_fwd(const fp8_block_norm_t* f, void* stream) {
  const char* who = "fp8_block_norm_fwd";
  FP8GB_TRY(check_norm(f, who));
  if ((f->hq == nullptr) != (f->hsf == nullptr)) return fail(FP8_ERR_INVALID_ARG, "%s: codes and their scales go together", who);
  if (f->hq != nullptr && !known(static_cast<fp4_format_t>(f->h_fmt)))
    return fail(FP8_ERR_INVALID_ARG, "%s: unknown format %d", who, (int)f->h_fmt);
  if (f->hq != nullptr && f->h_fmt != FP4_NVFP4 && f->h_scale != nullptr)
    return fail(FP8_ERR_INVALID_ARG, "%s: MXFP4 has no tensor scale", who);
  const bool empty = f->tokens == 0 || f->width == 0;
  if (!empty && f->r == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null r", who);
  if (!empty && f->r_out == nullptr && f->h == nullptr && f->hq == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: no output", who);
  FP8GB_TRY(check_matrix(f->h, f->ld_h, f->tokens, f->width, f->block_dt == FP8_DT_F32 ? 4 : 2, who, "h"));
  if (!aligned16(f->hq) || !aligned16(f->hsf)) return fail(FP8_ERR_ALIGNMENT, "%s: hq and hsf must be 16-byte aligned", who);
  if (!aligned_to(f->h_scale, 4)) return fail(FP8_ERR_ALIGNMENT, "%s: h_scale is not aligned to its elements", who);
  if (f->hq != nullptr && f->width % 32 != 0) return fail(FP8_ERR_UNSUPPORTED, "%s: hq needs width %% 32 == 0", who);
  if (f->r_out == f->r && f->r != nullptr && f->ld_r_out != f->ld_r && f->tokens > 1)
    return fail(FP8_ERR_INVALID_ARG, "%s: r_out is r with another leading dimension", who);
  if (empty) return FP8_OK;
  return done(launch_norm_fwd(to_fwd(f), static_cast<cudaStream_t>(stream)), who);
}

int64_t fp8_block_norm_bwd_workspace_bytes(const fp8_block_norm_t* f, const fp8_block_norm_grad_t* b) {
  const char* who = "fp8_block_norm_bwd_workspace_bytes";
  if (check_norm(f, who) != FP8_OK) return -1;
  if (b == nullptr) {
    fail(FP8_ERR_INVALID_ARG, "%s: null gradients", who);
    return -1;
  }
  if (check_device(who) != FP8_OK) return -1;
  return norm_bwd_workspace_bytes(to_fwd(f));
}

fp8_status_t fp8_block_norm_bwd(const fp8_block_norm_t* f, const fp8_block_norm_grad_t* b, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  const char* who = "fp8_block_norm_bwd";
  FP8GB_TRY(check_norm(f, who));
  if (b == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: null gradients", who);
  const bool empty = f->tokens == 0 || f->width == 0;
  if (!empty && b->dh == nullptr && b->dr_out == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: no gradient comes in", who);
  if (!empty && f->pre != FP8_NORM_NONE && b->dh != nullptr && (f->r_out == nullptr || f->stat_pre == nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: the norm before the next block needs r_out and stat_pre", who);
  if (!empty && f->post != FP8_NORM_NONE && f->stat_post == nullptr)
    return fail(FP8_ERR_INVALID_ARG, "%s: the norm after the block needs stat_post", who);
  if (!empty && b->dres_scale != nullptr && f->r == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: dres_scale needs r", who);
  if (b->dgate != nullptr && f->gate == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: dgate without a gate", who);
  if (!empty && b->do_ != nullptr && f->o == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: do without o", who);
  if (f->pre == FP8_NORM_NONE && (b->dw_pre != nullptr || b->db_pre != nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: dw_pre or db_pre without a norm before the next block", who);
  if (f->post == FP8_NORM_NONE && (b->dw_post != nullptr || b->db_post != nullptr))
    return fail(FP8_ERR_INVALID_ARG, "%s: dw_post or db_post without a norm after the block", who);
  const int64_t ss = f->stream_dt == FP8_DT_F32 ? 4 : 2, bs = f->block_dt == FP8_DT_F32 ? 4 : 2;
  FP8GB_TRY(check_matrix(b->dh, b->ld_dh, f->tokens, f->width, bs, who, "dh"));
  FP8GB_TRY(check_matrix(b->dr_out, b->ld_dr_out, f->tokens, f->width, ss, who, "dr_out"));
  FP8GB_TRY(check_matrix(b->dr, b->ld_dr, f->tokens, f->width, ss, who, "dr"));
  FP8GB_TRY(check_matrix(b->do_, b->ld_do, f->tokens, f->width, bs, who, "do"));
  const void* vec[] = {b->dgate, b->dres_scale, b->dw_post, b->db_post, b->dw_pre, b->db_pre};
  for (const void* v : vec) FP8GB_TRY(check_vector(v, who, "a gradient"));
  if (b->dr == b->dr_out && b->dr != nullptr && b->ld_dr != b->ld_dr_out && f->tokens > 1)
    return fail(FP8_ERR_INVALID_ARG, "%s: dr is dr_out with another leading dimension", who);
  if (workspace_bytes < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative workspace size", who);
  if (!aligned16(workspace)) return fail(FP8_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", who);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) {  // sums over no tokens
    float* out[] = {b->dw_post, b->db_post, b->dw_pre, b->db_pre};
    cudaError_t e = cudaSuccess;
    for (float* p : out)
      if (p != nullptr && f->width > 0 && e == cudaSuccess) e = cudaMemsetAsync(p, 0, f->width * 4, s);
    if (b->dres_scale != nullptr && e == cudaSuccess) e = cudaMemsetAsync(b->dres_scale, 0, 4, s);
    return done(e, who);
  }
  const NormFwd nf = to_fwd(f);
  const int64_t need = norm_bwd_workspace_bytes(nf);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(FP8_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who, (long long)(workspace ? workspace_bytes : 0), (long long)need);
  NormBwd nb{};
  nb.dh = b->dh;
  nb.dr_out = b->dr_out;
  nb.dr = b->dr;
  nb.dO = b->do_;
  nb.ld_dh = b->ld_dh;
  nb.ld_dr_out = b->ld_dr_out;
  nb.ld_dr = b->ld_dr;
  nb.ld_do = b->ld_do;
  nb.dgate = b->dgate;
  nb.dres_scale = b->dres_scale;
  nb.dw_post = b->dw_post;
  nb.db_post = b->db_post;
  nb.dw_pre = b->dw_pre;
  nb.db_pre = b->db_pre;
  return done(launch_norm_bwd(nf, nb, workspace, s), who);
}

}  // extern "C"
