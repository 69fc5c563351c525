"""An infinite gate where there is no bias after the block: r' is infinite there, not NaN, whichever kernel runs and whether or
not the next norm has a bias."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("T,D", [(5, 1024), (1300, 1024), (1300, 4096), (3, 16416)])
@pytest.mark.parametrize("bias", [False, True])
def test_infinite_gate(g, T, D, bias):
    gen = torch.Generator("cuda").manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    r, o, gate, w, b = n(T, D).bfloat16(), n(T, D).bfloat16(), n(1, D).bfloat16(), n(D), n(D)
    o[o == 0] = 1.0
    gate[0, 5] = float("inf")
    r_out, h = torch.zeros_like(r), torch.zeros_like(r)
    f = g.block_norm(T, D, g.FP8_DT_BF16, g.FP8_DT_BF16, post=g.FP8_NORM_RMS, pre=g.FP8_NORM_RMS, r=r, o=o, gate=gate, gate_rows=T, w_pre=w, b_pre=b if bias else None,
                     r_out=r_out, h=h)
    g.fp8_block_norm_fwd(f)
    torch.cuda.synchronize()
    assert torch.equal(r_out[:, 5].float(), torch.sign(o[:, 5].float()) * float("inf"))
    rest = torch.arange(D, device="cuda") != 5
    assert torch.isfinite(r_out[:, rest].float()).all()
    # 1 / root is 0: the other columns' h is the bias alone
    want = (b if bias else torch.zeros_like(b)).bfloat16()[rest]
    assert (h[:, rest].float() == want.float()).all()
