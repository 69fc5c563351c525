"""A gate's checks do not depend on how large gate_rows says "all tokens" is. On CPU: every call is refused before it touches
the GPU, device addresses are made-up numbers."""
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("host-side checks only: made-up device addresses", allow_module_level=True)

A, B, C, ODD = 0x10000, 0x20000, 0x30000, 0x10001


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("tokens", [1, 2, 4, 16384])
@pytest.mark.parametrize("rows", [16384, 1 << 40, (1 << 63) - 2, (1 << 63) - 1])
def test_a_gate_that_is_not_aligned(g, tokens, rows):
    f = g.block_norm(tokens, 64, 0, 0, r=A, ld_r=64, o=B, ld_o=64, gate=ODD, ld_gate=64, gate_rows=rows, r_out=C, ld_r_out=64)
    b = g.block_norm_grad(dr_out=A, ld_dr_out=64, dgate=C)
    for call in (lambda: g.fp8_block_norm_fwd(f), lambda: g.fp8_block_norm_bwd(f, b, A, 1 << 40), lambda: g.fp8_block_norm_bwd_workspace_bytes(f, b)):
        with pytest.raises(g.Fp8Error) as e:
            call()
        assert "gate is not aligned" in str(e.value)


def test_the_pitch_of_several_gates(g):
    f = g.block_norm(5, 64, 0, 0, r=A, ld_r=64, o=B, ld_o=64, gate=A, ld_gate=63, gate_rows=4, r_out=C, ld_r_out=64)
    with pytest.raises(g.Fp8Error) as e:
        g.fp8_block_norm_fwd(f)
    assert "ld of gate" in str(e.value)
