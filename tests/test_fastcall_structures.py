"""The C binding takes its structures by their class, as the ctypes wrappers do: blocks exchanged, buffers of other things and short
ones are refused before the library reads them. No GPU."""
import ctypes

import numpy as np
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


def wrong_type(g, name, *args, **kw):
    for fn in (g._by_ctypes[name], getattr(g, name)):
        with pytest.raises((TypeError, AttributeError, ctypes.ArgumentError)):
            fn(*args, **kw)


class Holder:
    def __init__(self, c):
        self.c = c


def test_other_structures_and_buffers(g):
    st = g.fp8_tensor_state_t(S, S, S, S, S, S, 16)
    f = g.block_norm(4, 64, 0, 0, r=A, ld_r=64, r_out=B, ld_r_out=64, stat_pre=S)
    b = g.block_norm_grad(dh=A, ld_dh=64, dr=C, ld_dr=64)
    others = [bytes(512), bytearray(512), memoryview(bytes(512)), np.zeros(512, dtype=np.uint8), (ctypes.c_char * 512)(), object(), "state", 1.5]
    for x in others + [st, b, Holder(st), Holder(f), Holder(bytes(512))]:
        wrong_type(g, "fp8_block_norm_fwd", x)
        wrong_type(g, "fp8_block_norm_bwd", x, b, None, 0)
    for x in others + [st, f, Holder(b)]:
        wrong_type(g, "fp8_block_norm_bwd", f, x, None, 0)
    for x in others + [f, b, Holder(f), Holder(bytes(512))]:
        wrong_type(g, "fp4_quantize", None, 0, 64, 64, 0, 0, x, None, None)  # (nothing to do otherwise)


def test_what_is_taken(g):
    st = g.fp8_tensor_state_t(0, 0, 0, S, S, S, 0)

    class Own(g.fp8_tensor_state_t):
        pass

    class Made:
        @property
        def c(self):  # a new one each time, held by nothing else
            return g.fp8_tensor_state_t(0, 0, 0, S, S, S, 0)

    for x in (st, Holder(st), Made(), Own(0, 0, 0, S, S, S, 0)):
        with pytest.raises(g.Fp8Error) as e:
            g.fp4_quantize(A, 16, 16, 16, 0, 0, x, B, C)
        assert "null scale" in str(e.value)
    for fn in (lambda: g.fp8_block_norm_fwd(None), lambda: g.fp8_block_norm_bwd(g.block_norm(1, 8, 0, 0), None, None, 0)):
        with pytest.raises(g.Fp8Error) as e:
            fn()
        assert "null" in str(e.value)
