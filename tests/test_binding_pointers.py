"""What the binding takes for a device pointer: None, an address, a tensor. Host buffers are refused; ctypes alone would pass their
host addresses on. No GPU: made-up addresses, and every call is refused or would be."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("host-side checks only: made-up device addresses", allow_module_level=True)

A, B, C = 0x10000, 0x20000, 0x30000


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("x", [b"codes" * 16, "codes", bytearray(64), ctypes.c_void_p(A), (ctypes.c_char * 64)(), 1.0, object()], ids=lambda x: type(x).__name__)
def test_host_buffers(g, x):
    dequantize = [getattr(g, "fp4_dequantize")] + ([g._by_ctypes["fp4_dequantize"]] if g._fastcall is not None else [])
    calls = [lambda f=f: f(x, B, 1, 8, 0, None, C, 0, 8) for f in dequantize]
    calls += [lambda: g.fp8_scaled_mm(x, 0, B, 0, 16, 16, 16, 16, 16, 0, A, A, C, 16), lambda: g.fp8_linear_bwd_noalloc(x, 16, 16, 16, A, None, A, None, None, 0, A, A),
              lambda: g.mm_problem(x, 0, B, 0, 16, 16, 16, 16, 16, A, A, C, 16), lambda: g.block_norm(1, 8, 0, 0, r=x, ld_r=8), lambda: g.block_norm_grad(dh=x, ld_dh=8)]
    for call in calls:
        with pytest.raises((AttributeError, TypeError)):
            call()


def test_what_is_taken(g):
    t = torch.zeros(8)
    assert g._ptr(None) is None and g._ptr(A) == A and g._ptr(t) == t.data_ptr()
