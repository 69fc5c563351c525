"""Refusals of the 4-bit and block-norm entry points, on CPU: every call below is refused before it
touches the GPU. Device addresses are made-up numbers; nothing is dereferenced."""
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("host-side checks only: made-up device addresses", allow_module_level=True)

A, B, C, S, ODD = 0x10000, 0x20000, 0x30000, 0x40000, 0x10001


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def refused(g, status, who, fn, *args, **kw):
    with pytest.raises(g.Fp8Error) as e:
        fn(*args, **kw)
    assert e.value.status == status, (e.value.status, str(e.value))
    assert who in str(e.value), str(e.value)


def test_sizes(g):
    assert [g.fp4_row_bytes(k) for k in (0, 1, 32, 33, 4096)] == [0, 16, 16, 32, 2048]
    assert g.fp4_scale_bytes(g.FP4_NVFP4, 1, 1) == 512 and g.fp4_scale_bytes(g.FP4_NVFP4, 129, 65) == 2048
    assert g.fp4_scale_bytes(g.FP4_MXFP4, 128, 128) == 512 and g.fp4_scale_bytes(g.FP4_MXFP4, 128, 129) == 1024
    for bad in ((2, 1, 1), (0, -1, 1), (0, 1, -1)):
        with pytest.raises(g.Fp8Error):
            g.fp4_scale_bytes(*bad)
    with pytest.raises(g.Fp8Error):
        g.fp4_row_bytes(-1)


def test_quantize(g):
    q = g.fp4_quantize
    st = g.fp8_tensor_state_t(S, S, S, S, S, S, 16)
    inv, al, un = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_ALIGNMENT, g.FP8_ERR_UNSUPPORTED
    refused(g, inv, "negative", q, A, -1, 16, 16, 0, 0, None, B, C)
    refused(g, inv, "format", q, A, 16, 16, 16, 2, 0, None, B, C)
    refused(g, inv, "scaling mode", q, A, 16, 16, 16, 0, 2, None, B, C)
    refused(g, inv, "together", q, A, 16, 16, 16, 0, 0, None, B, None)
    refused(g, inv, "together", q, A, 16, 16, 16, 0, 0, None, B, C, None, S)
    refused(g, inv, "no output", q, A, 16, 16, 16, 0, 0, None, None, None)
    refused(g, inv, "null input", q, None, 16, 16, 16, 0, 0, None, B, C)
    refused(g, inv, "ld", q, A, 16, 16, 15, 0, 0, None, B, C)
    refused(g, inv, "MXFP4", q, A, 16, 16, 16, 1, 0, st, B, C)
    refused(g, inv, "delayed", q, A, 16, 16, 16, 0, 1, None, B, C)
    refused(g, inv, "history", q, A, 16, 16, 16, 0, 1, g.fp8_tensor_state_t(0, 0, S, S, S, S, 0), B, C)
    refused(g, inv, "null scale", q, A, 16, 16, 16, 0, 0, g.fp8_tensor_state_t(0, 0, 0, S, S, S, 0), B, C)
    refused(g, al, "16-byte", q, A, 16, 16, 16, 0, 0, None, ODD, C)
    refused(g, al, "16-byte", q, A, 16, 16, 16, 0, 0, None, None, None, B, B + 8)
    refused(g, al, "elements", q, ODD, 16, 16, 16, 0, 0, None, B, C)
    refused(g, un, "2^31", q, A, 1 << 31, 16, 16, 0, 0, None, B, C)


def test_dequantize(g):
    d = g.fp4_dequantize
    inv, al, un = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_ALIGNMENT, g.FP8_ERR_UNSUPPORTED
    refused(g, inv, "negative", d, A, B, 1, -1, 0, None, C, 0, 8)
    refused(g, inv, "format", d, A, B, 1, 8, 5, None, C, 0, 8)
    refused(g, inv, "type", d, A, B, 1, 8, 0, None, C, 2, 8)
    refused(g, inv, "ldy", d, A, B, 1, 8, 0, None, C, 0, 7)
    refused(g, inv, "null", d, A, None, 1, 8, 0, None, C, 0, 8)
    refused(g, al, "16-byte", d, A + 8, B, 1, 8, 0, None, C, 0, 8)
    refused(g, al, "elements", d, A, B, 1, 8, 0, None, C + 2, 1, 8)
    refused(g, un, "2^31", d, A, B, 1, 1 << 31, 0, None, C, 0, 1 << 31)


def test_scaled_mm(g):
    mm = g.fp4_scaled_mm
    inv, al, un = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_ALIGNMENT, g.FP8_ERR_UNSUPPORTED
    refused(g, inv, "negative", mm, A, S, B, S, -1, 16, 16, 0, None, None, C, 0, 16)
    refused(g, inv, "format", mm, A, S, B, S, 16, 16, 16, 9, None, None, C, 0, 16)
    refused(g, inv, "type", mm, A, S, B, S, 16, 16, 16, 0, None, None, C, 9, 16)
    refused(g, inv, "ldc", mm, A, S, B, S, 16, 17, 16, 0, None, None, C, 0, 16)
    refused(g, inv, "null C", mm, A, S, B, S, 16, 16, 16, 0, None, None, None, 0, 16)
    refused(g, inv, "null A", mm, A, None, B, S, 16, 16, 16, 0, None, None, C, 0, 16)
    refused(g, al, "16-byte", mm, A, S, ODD, S, 16, 16, 16, 0, None, None, C, 0, 16)
    refused(g, al, "ldc", mm, A, S, B, S, 16, 16, 16, 0, None, None, C, 0, 20)
    refused(g, al, "ldc", mm, A, S, B, S, 16, 16, 16, 0, None, None, C, 1, 18)
    refused(g, al, "elements", mm, A, S, B, S, 16, 16, 16, 0, S + 1, None, C, 0, 16)
    refused(g, un, "2^31", mm, A, S, B, S, 1 << 31, 16, 16, 0, None, None, C, 0, 16)


def test_norm_forward(g):
    inv, al, un = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_ALIGNMENT, g.FP8_ERR_UNSUPPORTED
    M = dict(r=A, ld_r=64, r_out=B, ld_r_out=64)

    def f(status, who, tokens=4, width=64, sdt=0, bdt=0, **kw):
        refused(g, status, who, lambda: g.fp8_block_norm_fwd(g.block_norm(tokens, width, sdt, bdt, **{**M, **kw})))

    f(inv, "negative", tokens=-1)
    f(inv, "unknown type", sdt=2)
    f(inv, "unknown norm", pre=3)
    f(inv, "eps", eps=-1.0)
    f(inv, "eps", eps=float("nan"))
    f(un, "2^31", width=1 << 31, ld_r=1 << 31, ld_r_out=1 << 31)
    f(inv, "gate_rows", o=C, ld_o=64, gate=S, ld_gate=64)
    f(inv, "w_post", w_post=S)
    f(inv, "w_pre", pre=0, w_pre=S)
    f(inv, "without o", post=1)
    f(inv, "without o", gate=S, ld_gate=64, gate_rows=1)
    f(inv, "ld of r", ld_r=63)
    f(inv, "ld of o", o=C, ld_o=3)
    f(al, "r is not aligned", r=ODD)
    f(al, "h is not aligned", bdt=1, h=C + 2, ld_h=64)
    f(al, "parameter", w_pre=S + 2)
    f(al, "statistics", stat_pre=S + 4)
    f(inv, "null r", r=None)
    f(inv, "no output", r_out=None)
    f(inv, "together", hq=S)
    f(inv, "unknown format", hq=S, hsf=C, h_fmt=4)
    f(inv, "MXFP4", hq=S, hsf=C, h_fmt=1, h_scale=S)
    f(al, "hq", hq=S + 8, hsf=C)
    f(un, "width % 32", width=48, hq=S, hsf=C)
    f(inv, "another leading dimension", r_out=A, ld_r_out=128)
    with pytest.raises(TypeError):
        g.block_norm(1, 1, 0, 0, nothing=1)


def test_norm_backward(g):
    inv, al = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_ALIGNMENT
    F = dict(r=A, ld_r=64, r_out=B, ld_r_out=64, stat_pre=S)
    G = dict(dh=A, ld_dh=64, dr=C, ld_dr=64)

    def f(status, who, ws=S, n=1 << 40, fw=None, kind=None, **kw):
        a = g.block_norm(4, 64, 0, 0, **(kind or {}), **{**F, **(fw or {})})
        refused(g, status, who, lambda: g.fp8_block_norm_bwd(a, g.block_norm_grad(**{**G, **kw}), ws, n))

    f(inv, "no gradient", dh=None)
    f(inv, "needs r_out", fw=dict(r_out=None))
    f(inv, "needs r_out", fw=dict(stat_pre=None))
    f(inv, "stat_post", fw=dict(o=A, ld_o=64), kind=dict(post=1))
    f(inv, "dres_scale", fw=dict(r=None), dres_scale=S)
    f(inv, "dgate", dgate=S)
    f(inv, "do without o", do=S, ld_do=64)
    f(inv, "dw_post", dw_post=S)
    f(inv, "dw_pre", kind=dict(pre=0), dw_pre=S)
    f(inv, "ld of dh", ld_dh=1)
    f(al, "dr is not aligned", dr=ODD)
    f(al, "gradient", dw_pre=S + 1)
    f(al, "workspace", ws=S + 8)
    f(inv, "negative workspace", n=-1)
    f(inv, "needed", ws=None, n=0)
    f(inv, "needed", n=16)
    f(inv, "another leading dimension", dr_out=C, ld_dr_out=72)


def test_every_declared_fp4_function_is_exported_and_bound(g):
    import os
    import re
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8gb.h")).read()
    names = set(re.findall(r"\b(fp4_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", header, flags=re.S)))
    assert {"fp4_quantize", "fp4_dequantize", "fp4_scaled_mm", "fp4_row_bytes", "fp4_scale_bytes"} <= names
    assert all(hasattr(g.lib, n) and hasattr(g, n) for n in names)


def test_sizes_whose_tiles_end_past_32_bits(g):
    """A tile that a dimension ends in has to end below 2^31."""
    un, n = g.FP8_ERR_UNSUPPORTED, (1 << 31) - 1024
    refused(g, un, "2^31 - 1024", g.fp4_quantize, A, 1, n, n, 0, 0, None, B, C)
    refused(g, un, "2^31 - 1024", g.fp4_dequantize, A, B, n, 1, 0, None, C, 0, 1)
    refused(g, un, "2^31 - 1024", g.fp4_scaled_mm, A, S, B, S, 1, n, 16, 0, None, None, C, 0, 1 << 31)
    refused(g, un, "2^31 - 1024", lambda: g.fp8_block_norm_fwd(g.block_norm(n, 8, 0, 0, r=A, ld_r=8, r_out=B, ld_r_out=8)))
