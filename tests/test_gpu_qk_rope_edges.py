"""The rotation's gradient at the edges of its numbers, against the oracle in 64 bits: infinities in the incoming gradient of the last head, which
a warp's unused rows repeat; rows of very large and very small values (bounds: as in the rotation's tests)."""
import numpy as np
import pytest
import torch

from oracle import heads
from test_gpu_qk_rope import HALF, f64, fractions, pairs_magnitude

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("H", [1, 3, 5, 7, 13])
@pytest.mark.parametrize("D, inter, dt, off", [(64, False, torch.bfloat16, 0), (128, False, torch.bfloat16, 0), (256, True, torch.bfloat16, 0), (64, True, torch.float32, 0), (128, False, torch.bfloat16, 1)])
def test_an_infinity_in_the_last_head_and_dw(g, H, D, inter, dt, off):
    T = 2
    gen = torch.Generator(device="cuda").manual_seed(H)
    x, dy = (torch.zeros(T * H * D + off, dtype=dt, device="cuda") for _ in range(2))
    for t in (x, dy):
        t[off:] = torch.randn(T * H * D, generator=gen, device="cuda").to(dt)
    x, dy = (t[off:].view(T, H, D) for t in (x, dy))
    dy[1, H - 1, 5] = float("inf")
    turns, frac = fractions(g, D)
    pos = torch.tensor([1, 5], dtype=torch.int32, device="cuda")
    dw = torch.full((D,), 7.0, device="cuda")
    f = g.qk_rope(T, H, 0, D, D, int(dt == torch.float32), layout=int(inter), norm=1, eps=1e-5, turns=turns, pos=pos, q=x)
    b = g.qk_rope_grad(dq_out=dy, dq=torch.empty_like(dy), dw_q=dw)
    n = g.fp8_qk_rope_bwd_workspace_bytes(f, b)
    g.fp8_qk_rope_bwd(f, b, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    with np.errstate(invalid="ignore"):
        _, want = heads.backward(f64(dy), f64(x), None, 1e-5, heads.angle([1, 5], frac), inter)
    got = f64(dw)
    inf = np.isinf(want)
    assert inf.sum() == 2 and np.array_equal(got[inf], want[inf]) and np.all(np.isfinite(got[~inf]))  # (both members of the pair)


@pytest.mark.parametrize("D, inter, dt, off", [(64, False, torch.bfloat16, 0), (128, False, torch.float32, 0), (256, True, torch.bfloat16, 0), (64, True, torch.float32, 0), (128, False, torch.bfloat16, 1), (64, True, torch.float32, 1)])
@pytest.mark.parametrize("size, eps", [(1e16, 1e-5), (1e13, 0.0), (1e-14, 0.0), (1e-16, 0.0)])
def test_rows_of_every_size(g, D, inter, dt, off, size, eps):
    """Both kernels, without and with dw: 1 / root cubed would leave fp32's range here, nothing of the gradient does."""
    T, H = 5, 3
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, dy = (torch.zeros(T * H * D + off, dtype=dt, device="cuda") for _ in range(2))
    x[off:] = (size * torch.randn(T * H * D, generator=gen, device="cuda")).to(dt)
    dy[off:] = torch.randn(T * H * D, generator=gen, device="cuda").to(dt)
    x, dy = (t[off:].view(T, H, D) for t in (x, dy))
    w = 1 + 0.3 * torch.randn(D, generator=gen, device="cuda")
    turns, frac = fractions(g, D)
    f = g.qk_rope(T, H, 0, D, D, int(dt == torch.float32), layout=int(inter), norm=1, eps=eps, turns=turns, q=x, w_q=w)
    want, want_w = heads.backward(f64(dy), f64(x), f64(w), eps, heads.angle(range(T), frac), inter)
    e, d = (D / 32 + 24) * 2.0 ** -24, pairs_magnitude(f64(dy), D, inter)
    r = 1 / np.sqrt((f64(x) ** 2).mean(axis=-1, keepdims=True) + eps)
    z, dz = np.abs(f64(x) * r), d * np.abs(f64(w))
    bound = 2 * e * r * (dz + z * (dz * z).mean(axis=-1, keepdims=True)) + HALF[dt] * np.abs(want) + 1e-38
    for dw in (None, torch.full((D,), 7.0, device="cuda")):
        dx = torch.full_like(dy, 7.0)
        b = g.qk_rope_grad(dq_out=dy, dq=dx, dw_q=dw)
        n = g.fp8_qk_rope_bwd_workspace_bytes(f, b)
        g.fp8_qk_rope_bwd(f, b, torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n)
        assert np.all(np.abs(f64(dx) - want) <= bound)
        if dw is not None:
            assert np.all(np.abs(f64(dw) - want_w) <= (2 * e + (T * H + 64) * 2.0 ** -24) * (d * z).sum(axis=(0, 1)))
