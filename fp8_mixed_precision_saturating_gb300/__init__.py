"""Python binding of libfp8gb (the GB300 FP8 up-projection library).

Argument marshalling only: every entry point forwards to the C ABI of the same name
declared in include/fp8gb.h, and every step of the computation runs in the library's
CUDA kernels. Tensors may be passed as torch tensors (their ``data_ptr()`` is used) or as
raw integer device addresses; ``stream`` may be a torch.cuda.Stream, an integer handle
or None (the current torch stream when torch is importable, else the default stream).

There is no fallback: importing this package fails loudly when libfp8gb.so has not been
built (``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import ctypes
import importlib
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8gb.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libfp8gb.so is missing at {LIB_PATH}: build it first (fp8_mixed_precision_saturating_gb300._build.build())")

lib = ctypes.CDLL(LIB_PATH)
_fastcall = None

# enums (include/fp8gb.h)
FP8_OK, FP8_ERR_INVALID_ARG, FP8_ERR_UNSUPPORTED, FP8_ERR_ALIGNMENT, FP8_ERR_CUDA, FP8_ERR_TIMEOUT = range(6)
FP8_E4M3, FP8_E5M2 = 0, 1
FP8_GRAN_TENSOR, FP8_GRAN_TILE_1x128, FP8_GRAN_BLOCK_128x128, FP8_GRAN_MX_1x32 = 0, 1, 2, 3
FP8_SCALE_CURRENT, FP8_SCALE_DELAYED = 0, 1
FP4_NVFP4, FP4_MXFP4 = 0, 1
FP8_DT_BF16, FP8_DT_F32 = 0, 1
FP8_NORM_NONE, FP8_NORM_RMS, FP8_NORM_LAYER = 0, 1, 2
FP8_ROPE_HALF, FP8_ROPE_INTERLEAVED = 0, 1
FP8_ROPE_PLAIN, FP8_ROPE_LINEAR, FP8_ROPE_BASE, FP8_ROPE_PARTS, FP8_ROPE_PARTS_BY_INDEX = range(5)
FP8_KV_BF16, FP8_KV_MX_E4M3 = 0, 1


class fp8_tensor_state_t(ctypes.Structure):
    _fields_ = [
        ("amax_history", ctypes.c_void_p),
        ("hist_count", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("scale_inv", ctypes.c_void_p),
        ("amax_cur", ctypes.c_void_p),
        ("counters", ctypes.c_void_p),
        ("hist_len", ctypes.c_int32),
    ]


class fp8_block_norm_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "width")]
    _fields_ += [(n, ctypes.c_int32) for n in ("stream_dt", "block_dt", "post", "pre")]
    _fields_ += [("eps", ctypes.c_float)]
    _fields_ += [("r", ctypes.c_void_p), ("ld_r", ctypes.c_int64), ("o", ctypes.c_void_p), ("ld_o", ctypes.c_int64)]
    _fields_ += [("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64), ("gate_rows", ctypes.c_int64)]
    _fields_ += [(n, ctypes.c_void_p) for n in ("res_scale", "w_post", "b_post", "w_pre", "b_pre")]
    _fields_ += [("r_out", ctypes.c_void_p), ("ld_r_out", ctypes.c_int64), ("h", ctypes.c_void_p), ("ld_h", ctypes.c_int64)]
    _fields_ += [("hq", ctypes.c_void_p), ("hsf", ctypes.c_void_p), ("h_fmt", ctypes.c_int32), ("h_scale", ctypes.c_void_p)]
    _fields_ += [("stat_post", ctypes.c_void_p), ("stat_pre", ctypes.c_void_p)]


class fp8_block_norm_grad_t(ctypes.Structure):
    _fields_ = [("dh", ctypes.c_void_p), ("ld_dh", ctypes.c_int64), ("dr_out", ctypes.c_void_p), ("ld_dr_out", ctypes.c_int64)]
    _fields_ += [("dr", ctypes.c_void_p), ("ld_dr", ctypes.c_int64), ("do_", ctypes.c_void_p), ("ld_do", ctypes.c_int64)]
    _fields_ += [(n, ctypes.c_void_p) for n in ("dgate", "dres_scale", "dw_post", "db_post", "dw_pre", "db_pre")]


def _heads(*names):
    """Fields of head tensors: address, elements between tokens, elements between heads."""
    return [f for n in names for f in ((n, ctypes.c_void_p), ("ld_" + n, ctypes.c_int64), ("hs_" + n, ctypes.c_int64))]


class fp8_qk_rope_t(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64)]
    _fields_ += [(n, ctypes.c_int32) for n in ("q_heads", "k_heads", "head_dim", "rot_dims", "dt", "layout", "norm")]
    _fields_ += [("eps", ctypes.c_float), ("amplitude", ctypes.c_float), ("turns", ctypes.c_void_p), ("pos", ctypes.c_void_p)]
    _fields_ += _heads("q", "k", "v") + [("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p)] + _heads("q_out", "k_out")


class fp8_qk_rope_grad_t(ctypes.Structure):
    _fields_ = _heads("dq_out", "dk_out", "dq", "dk") + [("dw_q", ctypes.c_void_p), ("dw_k", ctypes.c_void_p)]


class fp8_kv_cache_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
    _fields_ += [(n, ctypes.c_int32) for n in ("format", "pages", "page_size", "heads", "head_dim")]
    _fields_ += [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride")]


class fp8_kv_batch_t(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("seqs", ctypes.c_int32), ("table_width", ctypes.c_int32), ("ld_table", ctypes.c_int64)]
    _fields_ += [(n, ctypes.c_void_p) for n in ("q_start", "kv_len", "page_table")]


class fp8_paged_attention_t(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float)] + _heads("q", "out") + [("lse", ctypes.c_void_p)]


class fp8_mm_problem_t(ctypes.Structure):
    _fields_ = [
        ("A", ctypes.c_void_p),
        ("fa", ctypes.c_int),
        ("B", ctypes.c_void_p),
        ("fb", ctypes.c_int),
        ("M", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("lda", ctypes.c_int64),
        ("ldb", ctypes.c_int64),
        ("scale_inv_a", ctypes.c_void_p),
        ("scale_inv_b", ctypes.c_void_p),
        ("C_bf16", ctypes.c_void_p),
        ("ldc", ctypes.c_int64),
        ("mn_major", ctypes.c_int32),
    ]


class fp8_quant_job_t(ctypes.Structure):
    _fields_ = [
        ("x_bf16", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("fmt", ctypes.c_int),
        ("mode", ctypes.c_int),
        ("st", ctypes.POINTER(fp8_tensor_state_t)),
        ("q_out", ctypes.c_void_p),
        ("qT_out", ctypes.c_void_p),
    ]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SP = ctypes.POINTER(fp8_tensor_state_t)
_MP = ctypes.POINTER(fp8_mm_problem_t)

_NP, _GP = ctypes.POINTER(fp8_block_norm_t), ctypes.POINTER(fp8_block_norm_grad_t)
_RP, _RGP = ctypes.POINTER(fp8_qk_rope_t), ctypes.POINTER(fp8_qk_rope_grad_t)
_CP, _BP, _AP = ctypes.POINTER(fp8_kv_cache_t), ctypes.POINTER(fp8_kv_batch_t), ctypes.POINTER(fp8_paged_attention_t)
_SIGS = {
    "fp8_quantize": [_P, _I64, _I64, _I64, _I, _I, _I, _SP, _P, _P, _P, _P],
    "fp8_scaled_mm": [_P, _I, _P, _I, _I64, _I64, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _P],
    "fp8_scaled_mm_ws": [_P, _I, _P, _I, _I64, _I64, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _P, _I64, _P],
    "fp8_scaled_mm_grouped": [_MP, ctypes.c_int32, _P, _I64, _P],
    "fp8_quantize_many": [ctypes.POINTER(fp8_quant_job_t), ctypes.c_int32, _P],
    "fp8_scaled_mm_quant": [_P, _I, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _I, _SP, _P, _P],
    "fp8_requantize_weights": [_P, _I64, _I64, _I, _I, _SP, _P, _P, _P, _P],
    "fp8_update_requantize_weights": [_P, _P, _I64, _I64, _I, _SP, _P, _P, _P],
    "fp8_linear_fwd": [_P, _I64, _I64, _I64, _P, _SP, _P, _SP, _I, _I, _P, _P, _P, _P, _P],
    "fp8_linear_bwd": [_P, _I64, _I64, _I64, _P, _SP, _P, _SP, _SP, _I, _P, _P, _P, _P, _P],
    "fp8_linear_bwd_noalloc": [_P, _I64, _I64, _I64, _P, _SP, _P, _SP, _SP, _I, _P, _P, _P],
    "fp8_linear_bwd_ws": [_P, _I64, _I64, _I64, _P, _SP, _P, _SP, _SP, _I, _P, _P, _P, _P, _P, _I64, _P],
    "fp8_linear_bwd_mn": [_P, _I64, _I64, _I64, _P, _SP, _P, _SP, _SP, _I, _P, _P, _P, _P, _I64, _P],
    "fp8_scaled_mm_t": [_P, _I, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _P],
    "fp4_quantize": [_P, _I64, _I64, _I64, _I, _I, _SP, _P, _P, _P, _P, _P],
    "fp4_dequantize": [_P, _P, _I64, _I64, _I, _P, _P, _I, _I64, _P],
    "fp4_scaled_mm": [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _I, _I64, _P],
    "fp8_block_norm_fwd": [_NP, _P],
    "fp8_block_norm_bwd": [_NP, _GP, _P, _I64, _P],
    "fp8_rope_turns": [ctypes.c_int32, ctypes.c_double, _I] + [ctypes.c_double] * 4 + [_P],
    "fp8_qk_rope_fwd": [_RP, _P],
    "fp8_qk_rope_bwd": [_RP, _RGP, _P, _I64, _P],
    "fp8_kv_append": [_RP, _CP, _BP, _P],
    "fp8_paged_attention": [_AP, _CP, _BP, _P, _I64, _P],
    "fp8_history_commit": [_SP, _P],
    "fp8_history_commit_many": [_SP, ctypes.c_int32, _P],
    "fp8_poll_device_error": [],
    "fp8_set_wait_limit_ns": [ctypes.c_ulonglong],
    "fp8_selftest_wait_timeout": [ctypes.c_ulonglong, _P],
    "fp8_get_last_error_detail": [ctypes.c_char_p, ctypes.c_size_t],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
lib.fp8_scaled_mm_grouped_workspace_bytes.argtypes = [_MP, ctypes.c_int32]
lib.fp8_scaled_mm_grouped_workspace_bytes.restype = ctypes.c_int64
lib.fp8_linear_bwd_workspace_bytes.argtypes = [_I64, _I64, _I64]
lib.fp8_linear_bwd_workspace_bytes.restype = ctypes.c_int64
lib.fp8_scaled_mm_workspace_bytes.argtypes = [_I64, _I64, _I64]
lib.fp8_scaled_mm_workspace_bytes.restype = ctypes.c_int64
lib.fp4_row_bytes.argtypes = [_I64]
lib.fp4_row_bytes.restype = ctypes.c_int64
lib.fp4_scale_bytes.argtypes = [_I, _I64, _I64]
lib.fp4_scale_bytes.restype = ctypes.c_int64
lib.fp8_block_norm_bwd_workspace_bytes.argtypes = [_NP, _GP]
lib.fp8_block_norm_bwd_workspace_bytes.restype = ctypes.c_int64
lib.fp8_qk_rope_bwd_workspace_bytes.argtypes = [_RP, _RGP]
lib.fp8_qk_rope_bwd_workspace_bytes.restype = ctypes.c_int64
lib.fp8_paged_attention_workspace_bytes.argtypes = [_AP, _CP, _BP]
lib.fp8_paged_attention_workspace_bytes.restype = ctypes.c_int64
lib.fp8_status_string.argtypes = [ctypes.c_int]
lib.fp8_status_string.restype = ctypes.c_char_p


class Fp8Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{fp8_status_string(status)}: {detail}")
        self.status = status
        self.detail = detail


def fp8_status_string(s: int) -> str:
    return lib.fp8_status_string(s).decode()


def fp8_get_last_error_detail() -> str:
    buf = ctypes.create_string_buffer(512)
    lib.fp8_get_last_error_detail(buf, 512)
    return buf.value.decode()


def _check(status: int) -> int:
    if status != FP8_OK:
        raise Fp8Error(status, fp8_get_last_error_detail())
    return status


def _ptr(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()  # (anything else, a host buffer above all, has none)


def _no_torch_stream():
    return None


def _find_current_stream():
    """A function that returns the raw handle of torch's current stream on the current device (None without a GPU).
    torch's raw-handle getter takes 0.2 us a call where torch.cuda.current_stream() takes 3, as much as a launch."""
    try:
        import torch
    except ImportError:
        return _no_torch_stream
    if not torch.cuda.is_available():
        return _no_torch_stream
    try:
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    except AttributeError:
        return lambda: torch.cuda.current_stream().cuda_stream
    torch.cuda.init()
    if _fastcall is not None:
        _fastcall.use_torch(raw, device)
    return lambda: raw(device())


_current_stream = None


def _stream(s):
    if s is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _state(st):
    if st is None:
        return None
    if isinstance(st, fp8_tensor_state_t):
        return ctypes.byref(st)
    return ctypes.byref(st.c)


class TensorState:
    """Device buffers of one tensor role's scaling state, allocated with torch (plumbing).

    Fields mirror fp8_tensor_state_t: amax_history [hist_len] fp32, hist_count int32,
    scale, scale_inv, amax_cur fp32, counters [2] int64 (read as uint64)."""

    def __init__(self, hist_len: int = 16, device="cuda"):
        import torch
        self.hist_len = hist_len
        self.buf_f = torch.zeros(hist_len + 3, dtype=torch.float32, device=device)
        self.buf_i = torch.zeros(1, dtype=torch.int32, device=device)
        self.buf_c = torch.zeros(2, dtype=torch.int64, device=device)
        self.amax_history = self.buf_f[:hist_len]
        self.scale = self.buf_f[hist_len:hist_len + 1]
        self.scale_inv = self.buf_f[hist_len + 1:hist_len + 2]
        self.amax_cur = self.buf_f[hist_len + 2:hist_len + 3]
        self.hist_count = self.buf_i
        self.counters = self.buf_c
        self.c = fp8_tensor_state_t(
            self.amax_history.data_ptr(), self.hist_count.data_ptr(), self.scale.data_ptr(),
            self.scale_inv.data_ptr(), self.amax_cur.data_ptr(), self.counters.data_ptr(), hist_len)

    def reset(self):
        self.buf_f.zero_()
        self.buf_i.zero_()
        self.buf_c.zero_()

    def snapshot(self) -> dict:
        """Host copy of the state (synchronises)."""
        f = self.buf_f.cpu().numpy()
        h = self.hist_len
        return dict(hist=f[:h].copy(), scale=f[h], scale_inv=f[h + 1], amax_cur=f[h + 2],
                    count=int(self.buf_i.cpu()[0]), overflow=int(self.buf_c.cpu()[0]), underflow=int(self.buf_c.cpu()[1]))


# ---------------------------------------------------------------------------------------
# entry points (same names and argument order as the C ABI)
# ---------------------------------------------------------------------------------------
def fp8_quantize(x, rows, cols, ld, fmt, gran, mode, st, q_out, qT_out=None, unit_scale_inv=None, stream=None):
    return _check(lib.fp8_quantize(_ptr(x), rows, cols, ld, fmt, gran, mode, _state(st), _ptr(q_out), _ptr(qT_out),
                                   _ptr(unit_scale_inv), _stream(stream)))


def fp8_scaled_mm(A, fa, B, fb, M, N, K, lda, ldb, gran, scale_inv_a, scale_inv_b, C, ldc, stream=None):
    return _check(lib.fp8_scaled_mm(_ptr(A), fa, _ptr(B), fb, M, N, K, lda, ldb, gran, _ptr(scale_inv_a),
                                    _ptr(scale_inv_b), _ptr(C), ldc, _stream(stream)))


def fp8_scaled_mm_ws(A, fa, B, fb, M, N, K, lda, ldb, gran, scale_inv_a, scale_inv_b, C, ldc, workspace,
                     workspace_bytes, stream=None):
    return _check(lib.fp8_scaled_mm_ws(_ptr(A), fa, _ptr(B), fb, M, N, K, lda, ldb, gran, _ptr(scale_inv_a),
                                       _ptr(scale_inv_b), _ptr(C), ldc, _ptr(workspace), workspace_bytes,
                                       _stream(stream)))


def quant_job(x, rows, cols, ld, fmt, mode, st, q, qT):
    """One fp8_quant_job_t (per-tensor scale) for fp8_quantize_many; keeps st alive."""
    c = st if isinstance(st, fp8_tensor_state_t) else st.c
    j = fp8_quant_job_t(_ptr(x), rows, cols, ld, fmt, mode, ctypes.pointer(c), _ptr(q), _ptr(qT))
    j._keep = st
    return j


def fp8_quantize_many(jobs, stream=None):
    arr = (fp8_quant_job_t * len(jobs))(*jobs)
    return _check(lib.fp8_quantize_many(arr, len(jobs), _stream(stream)))


def mm_problem(A, fa, B, fb, M, N, K, lda, ldb, scale_inv_a, scale_inv_b, C, ldc, mn_major=0):
    """One fp8_mm_problem_t (per-tensor scales) for fp8_scaled_mm_grouped."""
    return fp8_mm_problem_t(_ptr(A), fa, _ptr(B), fb, M, N, K, lda, ldb, _ptr(scale_inv_a), _ptr(scale_inv_b),
                            _ptr(C), ldc, mn_major)


def fp8_scaled_mm_grouped(problems, workspace=None, workspace_bytes=0, stream=None):
    arr = (fp8_mm_problem_t * len(problems))(*problems)
    return _check(lib.fp8_scaled_mm_grouped(arr, len(problems), _ptr(workspace), workspace_bytes, _stream(stream)))


def fp8_scaled_mm_grouped_workspace_bytes(problems) -> int:
    arr = (fp8_mm_problem_t * len(problems))(*problems)
    n = lib.fp8_scaled_mm_grouped_workspace_bytes(arr, len(problems))
    if n < 0:
        raise Fp8Error(FP8_ERR_INVALID_ARG, fp8_get_last_error_detail())
    return n


def fp8_scaled_mm_workspace_bytes(M, N, K) -> int:
    n = lib.fp8_scaled_mm_workspace_bytes(M, N, K)
    if n < 0:
        raise Fp8Error(FP8_ERR_CUDA, "fp8_scaled_mm_workspace_bytes")
    return n


def fp8_scaled_mm_quant(A, fa, B, fb, M, N, K, lda, ldb, scale_inv_a, scale_inv_b, C, ldc, fc, c_st, Cq,
                        stream=None):
    return _check(lib.fp8_scaled_mm_quant(_ptr(A), fa, _ptr(B), fb, M, N, K, lda, ldb, _ptr(scale_inv_a),
                                          _ptr(scale_inv_b), _ptr(C), ldc, fc, _state(c_st), _ptr(Cq), _stream(stream)))


def fp8_requantize_weights(w_master, K, N, gran, mode, st, wq_kn, wqT_nk, block_scale_inv=None, stream=None):
    return _check(lib.fp8_requantize_weights(_ptr(w_master), K, N, gran, mode, _state(st), _ptr(wq_kn), _ptr(wqT_nk),
                                             _ptr(block_scale_inv), _stream(stream)))


def fp8_update_requantize_weights(w_master, delta, K, N, mode, st, wq_kn, wqT_nk, stream=None):
    return _check(lib.fp8_update_requantize_weights(_ptr(w_master), _ptr(delta), K, N, mode, _state(st), _ptr(wq_kn),
                                                    _ptr(wqT_nk), _stream(stream)))


def fp8_linear_fwd(x, M, K, N, wqT_nk, w_st, w_block_scale_inv, x_st, gran, mode, xq_save, xqT_save,
                   x_tile_scale_inv, y, stream=None):
    return _check(lib.fp8_linear_fwd(_ptr(x), M, K, N, _ptr(wqT_nk), _state(w_st), _ptr(w_block_scale_inv),
                                     _state(x_st), gran, mode, _ptr(xq_save), _ptr(xqT_save), _ptr(x_tile_scale_inv),
                                     _ptr(y), _stream(stream)))


def fp8_linear_bwd(dy, M, K, N, xqT_save, x_st, wq_kn, w_st, dy_st, mode, dyq_ws, dyqT_ws, dx, dw, stream=None):
    return _check(lib.fp8_linear_bwd(_ptr(dy), M, K, N, _ptr(xqT_save), _state(x_st), _ptr(wq_kn), _state(w_st),
                                     _state(dy_st), mode, _ptr(dyq_ws), _ptr(dyqT_ws), _ptr(dx), _ptr(dw),
                                     _stream(stream)))


def fp8_linear_bwd_ws(dy, M, K, N, xqT_save, x_st, wq_kn, w_st, dy_st, mode, dyq_ws, dyqT_ws, dx, dw, workspace,
                      workspace_bytes, stream=None):
    return _check(lib.fp8_linear_bwd_ws(_ptr(dy), M, K, N, _ptr(xqT_save), _state(x_st), _ptr(wq_kn), _state(w_st),
                                        _state(dy_st), mode, _ptr(dyq_ws), _ptr(dyqT_ws), _ptr(dx), _ptr(dw),
                                        _ptr(workspace), workspace_bytes, _stream(stream)))


def fp8_linear_bwd_mn(dy, M, K, N, xq_save, x_st, wq_kn, w_st, dy_st, mode, dyq_ws, dx, dw, workspace=None,
                      workspace_bytes=0, stream=None):
    return _check(lib.fp8_linear_bwd_mn(_ptr(dy), M, K, N, _ptr(xq_save), _state(x_st), _ptr(wq_kn), _state(w_st),
                                        _state(dy_st), mode, _ptr(dyq_ws), _ptr(dx), _ptr(dw), _ptr(workspace),
                                        workspace_bytes, _stream(stream)))


def fp8_scaled_mm_t(A, fa, B, fb, M, N, K, lda, ldb, scale_inv_a, scale_inv_b, C, ldc, workspace=None,
                    workspace_bytes=0, stream=None):
    return _check(lib.fp8_scaled_mm_t(_ptr(A), fa, _ptr(B), fb, M, N, K, lda, ldb, _ptr(scale_inv_a),
                                      _ptr(scale_inv_b), _ptr(C), ldc, _ptr(workspace), workspace_bytes,
                                      _stream(stream)))


def fp8_linear_bwd_workspace_bytes(M, K, N) -> int:
    n = lib.fp8_linear_bwd_workspace_bytes(M, K, N)
    if n < 0:
        raise Fp8Error(FP8_ERR_CUDA, "fp8_linear_bwd_workspace_bytes")
    return n


def fp8_linear_bwd_noalloc(dy, M, K, N, xqT_save, x_st, wq_kn, w_st, dy_st, mode, dx, dw, stream=None):
    """fp8_linear_bwd with the dy codes in the library's static device array (no scratch
    arguments, no allocation by the call); see include/fp8gb.h for the size limit."""
    return _check(lib.fp8_linear_bwd_noalloc(_ptr(dy), M, K, N, _ptr(xqT_save), _state(x_st), _ptr(wq_kn),
                                             _state(w_st), _state(dy_st), mode, _ptr(dx), _ptr(dw), _stream(stream)))


# ---- microscaled 4-bit operands --------------------------------------------------------
def fp4_row_bytes(K) -> int:
    """Bytes of one row of K 4-bit codes."""
    n = lib.fp4_row_bytes(K)
    if n < 0:
        raise Fp8Error(FP8_ERR_INVALID_ARG, "fp4_row_bytes: negative size")
    return n


def fp4_scale_bytes(fmt, MN, K) -> int:
    """Bytes of the scale atoms of a 4-bit operand [MN, K]."""
    n = lib.fp4_scale_bytes(fmt, MN, K)
    if n < 0:
        raise Fp8Error(FP8_ERR_INVALID_ARG, "fp4_scale_bytes: negative size or unknown format")
    return n


def fp4_quantize(x, rows, cols, ld, fmt, mode, st, q, sf, qT=None, sfT=None, stream=None):
    return _check(lib.fp4_quantize(_ptr(x), rows, cols, ld, fmt, mode, _state(st), _ptr(q), _ptr(sf), _ptr(qT),
                                   _ptr(sfT), _stream(stream)))


def fp4_dequantize(q, sf, MN, K, fmt, scale_inv, y, dt, ldy, stream=None):
    return _check(lib.fp4_dequantize(_ptr(q), _ptr(sf), MN, K, fmt, _ptr(scale_inv), _ptr(y), dt, ldy,
                                     _stream(stream)))


def fp4_scaled_mm(A, sfa, B, sfb, M, N, K, fmt, scale_inv_a, scale_inv_b, C, dt, ldc, stream=None):
    return _check(lib.fp4_scaled_mm(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), M, N, K, fmt, _ptr(scale_inv_a),
                                    _ptr(scale_inv_b), _ptr(C), dt, ldc, _stream(stream)))


# ---- the norms around a block ----------------------------------------------------------
_TYPES = {FP8_DT_BF16: "torch.bfloat16", FP8_DT_F32: "torch.float32"}


def _types_of(dt):
    return [_TYPES[dt]] if dt in _TYPES else []  # (an unknown one is refused by the call)


def _of_type(name, t, types):
    """A tensor's elements are what the library reads there (``types``: names of torch types, empty: not known here)."""
    if types and str(t.dtype) not in types:
        raise TypeError(f"{name}: {t.dtype}, expected {' or '.join(types)}")


def _matrix(name, t, rows, cols):
    """The leading dimension of a matrix given as a tensor, a vector being one row: rows of consecutive elements, at least
    ``rows`` x ``cols``."""
    if t.dim() not in (1, 2):
        raise ValueError(f"{name} has {t.dim()} dimensions: give it as a matrix, or its leading dimension too")
    n, m = (1, t.shape[0]) if t.dim() == 1 else t.shape
    if m > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row are {t.stride(-1)} apart, not next to each other")
    if n < rows or m < cols:
        raise ValueError(f"{name} is {tuple(t.shape)}, smaller than [{rows}, {cols}]")
    return t.stride(0) if n > 1 else max(m, 1)


def _vector(name, t, n):
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    if t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, fewer than {n}")


def _fill(c, names, given, checks):
    """Set the fields of an argument block. A matrix given as a tensor brings its own row pitch unless ld_<name> is given too.
    Tensors are looked at first: checks[name] = (types, rows or None for a vector, columns or elements)."""
    unknown = set(given) - set(names)
    if unknown:
        raise TypeError(f"{type(c).__name__} has no {', '.join(sorted(unknown))}")
    pointers = {n for n, t in c._fields_ if t is ctypes.c_void_p}
    for name, v in given.items():
        if name not in pointers:
            setattr(c, name, v)
            continue
        if hasattr(v, "data_ptr"):
            types, rows, cols = checks[name]
            ld = "ld_" + name.rstrip("_")
            _of_type(name, v, types)
            if rows is None:
                _vector(name, v, cols)
            elif ld not in given:
                setattr(c, ld, _matrix(name, v, rows, cols))
        setattr(c, name, _ptr(v))
    c._keep = given  # the tensors stay alive with the block
    return c


def block_norm(tokens, width, stream_dt, block_dt, post=FP8_NORM_NONE, pre=FP8_NORM_RMS, eps=1e-5, **tensors):
    """An fp8_block_norm_t: what a program keeps for the norms around one block. Keywords are the fields of
    the C struct (r, o, gate, gate_rows, res_scale, w_post, ..., stat_pre; include/fp8gb.h). A tensor's type, size and
    strides are checked here (a leading dimension that is given by hand is taken as it is)."""
    c = fp8_block_norm_t(tokens=tokens, width=width, stream_dt=stream_dt, block_dt=block_dt, post=post, pre=pre, eps=eps)
    stream, block, f32, u8 = _types_of(stream_dt), _types_of(block_dt), ["torch.float32"], ["torch.uint8"]
    fmt, gate_rows = tensors.get("h_fmt", FP4_NVFP4), tensors.get("gate_rows", 0)
    groups = -(-tokens // gate_rows) if gate_rows > 0 else 0
    checks = {"r": (stream, tokens, width), "r_out": (stream, tokens, width), "o": (block, tokens, width), "h": (block, tokens, width),
              "gate": (block, groups, width), "res_scale": (f32, None, 1), "h_scale": (f32, None, 1), "stat_post": (f32, None, 2 * tokens),
              "stat_pre": (f32, None, 2 * tokens), "hq": (u8, None, tokens * lib.fp4_row_bytes(width)), "hsf": (u8, None, lib.fp4_scale_bytes(fmt, tokens, width)),
              **{k: (f32, None, width) for k in ("w_post", "b_post", "w_pre", "b_pre")}}
    return _fill(c, [n for n, _ in fp8_block_norm_t._fields_[7:]], tensors, checks)


_GRADS = ("dh", "dr_out", "dr", "do_")


def block_norm_grad(**tensors):
    """An fp8_block_norm_grad_t; keywords are its fields, with ``do`` for ``do_``."""
    if "do" in tensors:
        tensors["do_"] = tensors.pop("do")
    checks = {n: (["torch.float32"], None, 1) for n, t in fp8_block_norm_grad_t._fields_ if t is ctypes.c_void_p}
    checks.update({n: (list(_TYPES.values()), 0, 0) for n in _GRADS})  # (which type and how large: fp8_block_norm_bwd_workspace_bytes)
    return _fill(fp8_block_norm_grad_t(), [n for n, _ in fp8_block_norm_grad_t._fields_], tensors, checks)


def _check_grads(f, b):
    """The tensors of a gradient block against the norm's sizes and types."""
    given, groups = getattr(b, "_keep", {}), -(-f.tokens // f.gate_rows) if f.gate_rows > 0 else 0
    for name, v in given.items():
        if not hasattr(v, "data_ptr"):
            continue
        if name in _GRADS:
            dt = f.block_dt if name in ("dh", "do_") else f.stream_dt
            _of_type(name, v, _types_of(dt))
            if "ld_" + name.rstrip("_") not in given:
                _matrix(name, v, f.tokens, f.width)
        else:
            _vector(name, v, groups * f.width if name == "dgate" else 1 if name == "dres_scale" else f.width)


def fp8_block_norm_fwd(f, stream=None):
    return _check(lib.fp8_block_norm_fwd(f, _stream(stream)))


def fp8_block_norm_bwd(f, b, workspace, workspace_bytes, stream=None):
    return _check(lib.fp8_block_norm_bwd(f, b, _ptr(workspace), workspace_bytes, _stream(stream)))


def fp8_block_norm_bwd_workspace_bytes(f, b) -> int:
    """Bytes of workspace; b's tensors are checked against f's sizes and types on the way."""
    if isinstance(f, fp8_block_norm_t) and isinstance(b, fp8_block_norm_grad_t):
        _check_grads(f, b)
    n = lib.fp8_block_norm_bwd_workspace_bytes(f, b)
    if n < 0:
        raise Fp8Error(FP8_ERR_INVALID_ARG, fp8_get_last_error_detail())
    return n


# ---- heads turned by their position, a paged cache, attention over it -------------------------
def fp8_rope_turns(rot_dims, base, kind, factor, original, low, high, turns):
    """turns: the address of rot_dims / 2 unsigned 64-bit numbers in host memory (rope_turns makes a tensor)."""
    return _check(lib.fp8_rope_turns(rot_dims, base, kind, factor, original, low, high, turns))


def rope_turns(rot_dims, base, kind=FP8_ROPE_PLAIN, factor=1.0, original=0.0, low=1.0, high=4.0, device="cuda"):
    """The frequencies of a rotation as fractions of a turn per position, an int64 tensor [rot_dims / 2] that holds the
    unsigned numbers of include/fp8gb.h; what a program keeps for all its layers."""
    import torch
    host = (ctypes.c_uint64 * max(rot_dims // 2, 1))()
    fp8_rope_turns(rot_dims, base, kind, factor, original, low, high, host)
    return torch.tensor(list((ctypes.c_int64 * len(host)).from_buffer(host))[: rot_dims // 2], dtype=torch.int64, device=device)


def _head_tensor(name, t, tokens, heads, dim):
    """Elements between two tokens and between two heads of a tensor [tokens, heads, dim]."""
    if t.dim() != 3:
        raise ValueError(f"{name} has {t.dim()} dimensions: give it as [tokens, heads, head_dim], or its ld and hs too")
    if t.shape[0] < tokens or t.shape[1] < heads or t.shape[2] < dim:
        raise ValueError(f"{name} is {tuple(t.shape)}, smaller than [{tokens}, {heads}, {dim}]")
    if dim > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a head are {t.stride(2)} apart, not next to each other")
    return t.stride(0), t.stride(1)


def _fill_heads(c, names, given, checks):
    """Set the fields of an argument block with head tensors. A tensor brings its strides unless ld_<name> and hs_<name> are
    given too. checks[name] = (types, (tokens, heads, dim)) or (types, elements of a vector)."""
    unknown = set(given) - set(names)
    if unknown:
        raise TypeError(f"{type(c).__name__} has no {', '.join(sorted(unknown))}")
    for name, v in given.items():
        if name not in checks:
            setattr(c, name, v)
            continue
        types, size = checks[name]
        if hasattr(v, "data_ptr"):
            _of_type(name, v, types)
            if not isinstance(size, tuple):
                _vector(name, v, size)
            elif "ld_" + name in given or "hs_" + name in given:
                if "ld_" + name not in given or "hs_" + name not in given:
                    raise TypeError(f"{name}: ld_{name} and hs_{name} go together")
            else:
                ld, hs = _head_tensor(name, v, *size)
                setattr(c, "ld_" + name, ld)
                setattr(c, "hs_" + name, hs)
        setattr(c, name, _ptr(v))
    c._keep = given
    return c


def qk_rope(tokens, q_heads, k_heads, head_dim, rot_dims, dt, layout=FP8_ROPE_HALF, norm=FP8_NORM_NONE, eps=1e-6, amplitude=1.0, **tensors):
    """An fp8_qk_rope_t: what a program keeps for the heads of one layer. Keywords are the fields of the C struct (turns, pos, q, k, v, w_q,
    w_k, q_out, k_out; include/fp8gb.h); head tensors are [tokens, heads, head_dim] views with any strides but the last."""
    c = fp8_qk_rope_t(tokens=tokens, q_heads=q_heads, k_heads=k_heads, head_dim=head_dim, rot_dims=rot_dims, dt=dt, layout=layout, norm=norm, eps=eps,
                      amplitude=amplitude)
    types, f32, q, k = _types_of(dt), ["torch.float32"], (tokens, q_heads, head_dim), (tokens, k_heads, head_dim)
    checks = {"turns": (["torch.int64", "torch.uint64"], rot_dims // 2), "pos": (["torch.int32"], tokens), "w_q": (f32, head_dim), "w_k": (f32, head_dim),
              "q": (types, q), "q_out": (types, q), "k": (types, k), "k_out": (types, k), "v": (types, k)}
    return _fill_heads(c, [n for n, _ in fp8_qk_rope_t._fields_[10:]], tensors, checks)


def qk_rope_grad(**tensors):
    """An fp8_qk_rope_grad_t; keywords are its fields."""
    types = list(_TYPES.values())
    checks = {n: (types, (0, 0, 0)) for n in ("dq_out", "dk_out", "dq", "dk")}
    checks.update({n: (["torch.float32"], 1) for n in ("dw_q", "dw_k")})  # (which type and how large: fp8_qk_rope_bwd_workspace_bytes)
    return _fill_heads(fp8_qk_rope_grad_t(), [n for n, _ in fp8_qk_rope_grad_t._fields_], tensors, checks)


def _check_rope_grads(f, b):
    """The tensors of a gradient block against the heads' sizes and types."""
    given = getattr(b, "_keep", {})
    for name, v in given.items():
        if not hasattr(v, "data_ptr"):
            continue
        if name in ("dw_q", "dw_k"):
            _vector(name, v, f.head_dim)
        else:
            _of_type(name, v, _types_of(f.dt))
            if "ld_" + name not in given:
                _head_tensor(name, v, f.tokens, f.q_heads if name.startswith("dq") else f.k_heads, f.head_dim)


def kv_cache(k, v, k_scale=None, v_scale=None):
    """An fp8_kv_cache_t of tensors [pages, heads, page_size, head_dim] (any strides but the last: keys and values alike): bf16, or
    uint8 codes with uint8 scales [pages, heads, page_size, head_dim / 32], contiguous."""
    if k.dim() != 4 or v.shape != k.shape or any(a != b for a, b, n in zip(k.stride(), v.stride(), k.shape) if n > 1):
        raise ValueError("k and v: [pages, heads, page_size, head_dim], of the same shape and strides")
    if k.shape[3] > 1 and k.stride(3) != 1:
        raise ValueError("k: the elements of a head are not next to each other")
    mx = k_scale is not None or v_scale is not None
    for name, t in (("k", k), ("v", v)):
        _of_type(name, t, ["torch.uint8"] if mx else ["torch.bfloat16"])
    pages, heads, page, dim = k.shape
    if mx:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None or tuple(t.shape) != (pages, heads, page, dim // 32) or not t.is_contiguous():
                raise ValueError(f"{name}: [pages, heads, page_size, head_dim / 32], contiguous")
            _of_type(name, t, ["torch.uint8"])
    c = fp8_kv_cache_t(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), FP8_KV_MX_E4M3 if mx else FP8_KV_BF16, pages, page, heads, dim, *k.stride()[:3])
    c._keep = (k, v, k_scale, v_scale)
    return c


def kv_batch(tokens, q_start, kv_len, page_table):
    """An fp8_kv_batch_t of int32 tensors q_start [seqs + 1], kv_len [seqs] and page_table [seqs, table_width]."""
    seqs = kv_len.numel()
    for name, t in (("q_start", q_start), ("kv_len", kv_len), ("page_table", page_table)):
        _of_type(name, t, ["torch.int32"])
    _vector("q_start", q_start, seqs + 1)
    _vector("kv_len", kv_len, seqs)
    if page_table.dim() != 2 or page_table.shape[0] != seqs:
        raise ValueError(f"page_table is {tuple(page_table.shape)}, not [{seqs}, table_width]")
    c = fp8_kv_batch_t(tokens, seqs, page_table.shape[1], _matrix("page_table", page_table, seqs, 0), q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr())
    c._keep = (q_start, kv_len, page_table)
    return c


def paged_attention(q_heads, scale, window=0, q=None, out=None, lse=None, **strides):
    """An fp8_paged_attention_t: bf16 head tensors q and out [tokens, q_heads, head_dim], lse [tokens, q_heads] fp32 or None. Sizes are
    checked against a cache and a batch by fp8_paged_attention_workspace_bytes."""
    bf = ["torch.bfloat16"]
    given = {n: v for n, v in (("q", q), ("out", out), ("lse", lse)) if v is not None}
    return _fill_heads(fp8_paged_attention_t(q_heads=q_heads, window=window, scale=scale), [n for n, _ in fp8_paged_attention_t._fields_[3:]], {**given, **strides},
                       {"q": (bf, (0, q_heads, 0)), "out": (bf, (0, q_heads, 0)), "lse": (["torch.float32"], 0)})


def _check_attention(a, c, b):
    given = getattr(a, "_keep", {})
    for name, v in given.items():
        if not hasattr(v, "data_ptr"):
            continue
        if name == "lse":
            _vector(name, v, b.tokens * a.q_heads)
        elif "ld_" + name not in given:
            _head_tensor(name, v, b.tokens, a.q_heads, c.head_dim)


def fp8_qk_rope_fwd(f, stream=None):
    return _check(lib.fp8_qk_rope_fwd(f, _stream(stream)))


def fp8_qk_rope_bwd(f, b, workspace, workspace_bytes, stream=None):
    return _check(lib.fp8_qk_rope_bwd(f, b, _ptr(workspace), workspace_bytes, _stream(stream)))


def fp8_qk_rope_bwd_workspace_bytes(f, b) -> int:
    """Bytes of workspace; b's tensors are checked against f's sizes and types on the way."""
    if isinstance(f, fp8_qk_rope_t) and isinstance(b, fp8_qk_rope_grad_t):
        _check_rope_grads(f, b)
    n = lib.fp8_qk_rope_bwd_workspace_bytes(f, b)
    if n < 0:
        raise Fp8Error(FP8_ERR_INVALID_ARG, fp8_get_last_error_detail())
    return n


def fp8_kv_append(f, cache, batch, stream=None):
    return _check(lib.fp8_kv_append(f, cache, batch, _stream(stream)))


def fp8_paged_attention(a, cache, batch, workspace, workspace_bytes, stream=None):
    return _check(lib.fp8_paged_attention(a, cache, batch, _ptr(workspace), workspace_bytes, _stream(stream)))


def fp8_paged_attention_workspace_bytes(a, cache, batch) -> int:
    """Bytes of workspace; a's tensors are checked against the cache's and the batch's sizes on the way."""
    if isinstance(a, fp8_paged_attention_t) and isinstance(cache, fp8_kv_cache_t) and isinstance(batch, fp8_kv_batch_t):
        _check_attention(a, cache, batch)
    n = lib.fp8_paged_attention_workspace_bytes(a, cache, batch)
    if n < 0:
        raise Fp8Error(FP8_ERR_INVALID_ARG, fp8_get_last_error_detail())
    return n


def fp8_history_commit(st, stream=None):
    return _check(lib.fp8_history_commit(_state(st), _stream(stream)))


def fp8_history_commit_many(states, stream=None):
    """Push the amaxes of several distinct states in one launch (at most 32)."""
    arr = (fp8_tensor_state_t * len(states))(*[st if isinstance(st, fp8_tensor_state_t) else st.c for st in states])
    return _check(lib.fp8_history_commit_many(arr, len(states), _stream(stream)))


def fp8_poll_device_error():
    return _check(lib.fp8_poll_device_error())


def fp8_set_wait_limit_ns(ns: int):
    return _check(lib.fp8_set_wait_limit_ns(ns))


def fp8_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    """Returns the raw status (FP8_ERR_TIMEOUT is the expected result)."""
    return lib.fp8_selftest_wait_timeout(limit_ns, _stream(stream))


# ---------------------------------------------------------------------------------------
# the same calls in C (csrc/fastcall.c), where the host could build them
# ---------------------------------------------------------------------------------------
try:
    _fastcall = importlib.import_module(__name__ + "._fastcall")
except ImportError:
    pass
if _fastcall is not None:
    _NAMES = ("fp4_quantize", "fp4_dequantize", "fp4_scaled_mm", "fp8_block_norm_fwd", "fp8_block_norm_bwd", "fp8_qk_rope_fwd", "fp8_qk_rope_bwd",
              "fp8_kv_append", "fp8_paged_attention")
    _fastcall.init(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _NAMES), _check, _stream,
                   (fp8_tensor_state_t, fp8_block_norm_t, fp8_block_norm_grad_t, fp8_qk_rope_t, fp8_qk_rope_grad_t, fp8_kv_cache_t, fp8_kv_batch_t,
                    fp8_paged_attention_t))
    _by_ctypes = {n: globals()[n] for n in _NAMES}  # (what a host without Python.h calls)
    globals().update({n: getattr(_fastcall, n) for n in _NAMES})
