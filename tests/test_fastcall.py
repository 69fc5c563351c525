"""The binding's C calls (csrc/fastcall.c) beside the ctypes wrappers of the same names: arguments by position and by
name, what is missing or too much, the same refusals. No GPU."""
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("host-side checks only: made-up device addresses", allow_module_level=True)

A, B, C, S = 0x10000, 0x20000, 0x30000, 0x40000


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    if m._fastcall is None:
        pytest.skip("no Python.h to build with")
    return m


def both(g, name):
    return g._by_ctypes[name], getattr(g, name)


def same_refusal(g, name, *args, **kw):
    said = []
    for fn in both(g, name):
        with pytest.raises(g.Fp8Error) as e:
            fn(*args, **kw)
        said.append((e.value.status, str(e.value)))
    assert said[0] == said[1]
    return said[0]


def test_same_refusals(g):
    st = g.fp8_tensor_state_t(0, 0, 0, S, S, S, 0)
    assert same_refusal(g, "fp4_quantize", A, -1, 16, 16, 0, 0, None, B, C)[0] == g.FP8_ERR_INVALID_ARG
    assert "null scale" in same_refusal(g, "fp4_quantize", A, 16, 16, 16, 0, 0, st, B, C)[1]
    assert "MXFP4" in same_refusal(g, "fp4_quantize", A, 16, 16, 16, 1, 0, st, B, C, None, None, 0)[1]
    assert "together" in same_refusal(g, "fp4_quantize", A, 16, 16, 16, 0, 0, None, None, None, sfT=B)[1]
    assert "ldy" in same_refusal(g, "fp4_dequantize", A, B, 1, 8, 0, None, C, 0, 7, stream=5)[1]
    assert "ldc" in same_refusal(g, "fp4_scaled_mm", A, S, B, S, 16, 17, 16, 0, None, None, C, 0, 16)[1]
    f = g.block_norm(4, 64, 0, 0, r=A, ld_r=64)
    assert "no output" in same_refusal(g, "fp8_block_norm_fwd", f)[1]
    f = g.block_norm(4, 64, 0, 0, r=A, ld_r=64, r_out=B, ld_r_out=64, stat_pre=S)
    b = g.block_norm_grad(dh=A, ld_dh=64, dr=C, ld_dr=64)
    assert "needed" in same_refusal(g, "fp8_block_norm_bwd", f, b, None, 0, stream=None)[1]
    for fn in both(g, "fp4_quantize"):
        assert fn(None, 0, 64, 64, 0, 0, None, None, None) == 0  # nothing to do


def test_calls_that_do_not_fit(g):
    for fn in both(g, "fp4_dequantize"):
        for args, kw in (((A, B, 1), {}), ((A, B, 1, 8, 0, None, C, 0, 8, None, 1), {}), ((A, B, 1, 8, 0, None, C, 0), {"nothing": 1}),
                         ((A, B, 1, 8, 0, None, C, 0, 8), {"ldy": 8})):
            with pytest.raises(TypeError):
                fn(*args, **kw)
    with pytest.raises((TypeError, OverflowError)):
        g.fp4_dequantize(A, B, 1, 8, 1 << 40, None, C, 0, 8)
    with pytest.raises((TypeError, AttributeError)):
        g.fp4_dequantize("codes", B, 1, 8, 0, None, C, 0, 8)
    with pytest.raises((TypeError, AttributeError)):
        g.fp8_block_norm_fwd(object())
