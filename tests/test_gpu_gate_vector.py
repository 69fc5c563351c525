"""A matrix of one row is read the same way whatever pitch it is given with: a gate that is a vector has the bits of a [1, D]
one, and a token that is a row of a wider matrix those of a compact one (the kernels' sums differ in their order, so
equal bits say that the same kernel ran)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def run(g, T, D, x, gate, block):
    """Forward and backward; every matrix as `block` lays it out."""
    new = lambda t: block(torch.full_like(t, 7.0))  # noqa: E731
    lds = lambda **m: {**m, **{"ld_" + k: v.stride(0) for k, v in m.items() if v.dim() == 2}}  # noqa: E731
    vec = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    x = {k: block(v) if v.dim() == 2 else v for k, v in x.items()}
    out, stat_post, stat_pre = dict(r_out=new(x["r"]), h=new(x["o"])), vec(T, 2), vec(T, 2)
    f = g.block_norm(T, D, g.FP8_DT_BF16, g.FP8_DT_BF16, post=g.FP8_NORM_RMS, pre=g.FP8_NORM_LAYER, gate=gate, ld_gate=gate.stride(0), gate_rows=T, w_post=x["w"],
                     w_pre=x["w"], b_pre=x["b"], res_scale=x["alpha"], stat_post=stat_post, stat_pre=stat_pre, **lds(r=x["r"], o=x["o"], **out))
    g.fp8_block_norm_fwd(f)
    back = dict(dr=new(x["r"]), do=new(x["o"]))
    sums = dict(dgate=vec(1, D), dres_scale=vec(1), dw_post=vec(D), dw_pre=vec(D), db_pre=vec(D))
    b = g.block_norm_grad(**lds(dh=x["dh"], dr_out=x["dr"], **back), **sums)
    n = g.fp8_block_norm_bwd_workspace_bytes(f, b)
    g.fp8_block_norm_bwd(f, b, torch.zeros(n, dtype=torch.uint8, device="cuda"), n)
    torch.cuda.synchronize()
    return {**out, **back, **sums, "stat_post": stat_post, "stat_pre": stat_pre}


def inputs(T, D):
    gen = torch.Generator("cuda").manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(r=n(T, D).bfloat16(), o=n(T, D).bfloat16(), dh=n(T, D).bfloat16(), dr=n(T, D).bfloat16(), w=n(D), b=n(D),
                alpha=torch.full((1,), 0.9, device="cuda")), n(1, D).bfloat16()


@pytest.mark.parametrize("T,D", [(60, 1024), (60, 4096), (1300, 1024), (1300, 4096), (20, 12288)])
def test_gate_as_a_vector(g, T, D):
    x, gate = inputs(T, D)
    want, got = run(g, T, D, x, gate, lambda t: t), run(g, T, D, x, gate.view(D), lambda t: t)
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("D", [768, 2048, 4096, 8192])
def test_one_token_of_an_odd_pitch(g, D):
    def apart(t):  # a row of a matrix whose rows are D + 1 elements apart, itself on 16 bytes
        return torch.cat([t.reshape(-1), t.new_zeros(1)]).as_strided((1, D), (D + 1, 1))

    for seed in range(8):
        x, gate = inputs(1, D)
        x["r"] = (x["r"].float() * (1 + seed)).bfloat16()
        want, got = run(g, 1, D, x, gate, lambda t: t), run(g, 1, D, x, gate, apart)
        for k in want:
            assert torch.equal(got[k], want[k]), k
