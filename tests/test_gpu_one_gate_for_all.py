"""A gate of more rows than there are tokens is one gate for all of them, up to the largest number that the argument
holds: the bits of a call that says `gate_rows = tokens`."""
import pytest
import torch

pytestmark = pytest.mark.gpu

MOST = (1 << 63) - 1


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def outputs(g, T, D, gate_rows, x):
    """Everything that the forward and the backward write."""
    like = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    vec = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    out = dict(r_out=like(x["r"]), h=like(x["o"]), stat_post=vec(T, 2), stat_pre=vec(T, 2))
    f = g.block_norm(T, D, g.FP8_DT_BF16, g.FP8_DT_BF16, post=g.FP8_NORM_LAYER, pre=g.FP8_NORM_RMS, r=x["r"], o=x["o"], gate=x["gate"], gate_rows=gate_rows,
                     res_scale=x["alpha"], w_post=x["w"], b_post=x["b"], w_pre=x["w"], **out)
    g.fp8_block_norm_fwd(f)
    back = dict(dr=like(x["r"]), do=like(x["o"]), dgate=vec(1, D), dres_scale=vec(1), dw_post=vec(D), db_post=vec(D), dw_pre=vec(D), db_pre=vec(D))
    b = g.block_norm_grad(dh=x["dh"], dr_out=x["dr"], **back)
    n = g.fp8_block_norm_bwd_workspace_bytes(f, b)
    g.fp8_block_norm_bwd(f, b, torch.zeros(n, dtype=torch.uint8, device="cuda"), n)
    torch.cuda.synchronize()
    return {**out, **back}


@pytest.mark.parametrize("T,D", [(1, 72), (2, 72), (3, 256), (4, 72), (50, 77), (700, 520), (1300, 1024), (40, 8200)])
def test_gate_rows_up_to_the_largest_number(g, T, D):
    gen = torch.Generator("cuda").manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = dict(r=n(T, D).bfloat16(), o=n(T, D).bfloat16(), gate=n(1, D).bfloat16(), dh=n(T, D).bfloat16(), dr=n(T, D).bfloat16(), w=n(D), b=n(D),
             alpha=torch.full((1,), 0.9, device="cuda"))
    want = outputs(g, T, D, T, x)
    for rows in (T + 1, 1 << 40, MOST - 1, MOST):
        got = outputs(g, T, D, rows, x)
        for k in want:
            assert torch.equal(got[k], want[k]), (rows, k)
