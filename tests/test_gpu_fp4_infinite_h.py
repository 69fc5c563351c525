"""An infinity in a row that the norm writes in 4 bits counts as the largest finite bf16 in its group's magnitude, also under a
tensor scale so small that this is not past the largest group scale: the group's other elements keep their codes."""
import numpy as np
import pytest
import torch

from oracle import fp4

from gpu_util import host_u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("T,D", [(2, 64), (1300, 1056), (2, 16416)])
@pytest.mark.parametrize("scale", [1e-36, 2e-37, 1.0])
def test_infinity_under_a_small_scale(g, T, D, scale):
    gen = torch.Generator("cuda").manual_seed(D)
    r = torch.randn(T, D, generator=gen, device="cuda") * 5e37
    r[0, 3] = float("inf")
    r[T - 1, 40] = float("-inf")
    q = torch.full((T, g.fp4_row_bytes(D)), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((g.fp4_scale_bytes(fp4.NV, T, D),), 0xA5, dtype=torch.uint8, device="cuda")
    h = torch.empty(T, D, device="cuda")
    f = g.block_norm(T, D, g.FP8_DT_F32, g.FP8_DT_F32, pre=g.FP8_NORM_NONE, r=r, o=torch.zeros(T, D, device="cuda"), h=h, hq=q, hsf=sf, h_fmt=fp4.NV,
                     h_scale=torch.tensor([scale], device="cuda"))
    g.fp8_block_norm_fwd(f)
    torch.cuda.synchronize()
    assert torch.equal(h, r)
    want_q, want_sf = fp4.pack(*fp4.quantize(h.cpu().numpy(), fp4.NV, np.float32(scale)), fp4.NV)
    assert np.array_equal(host_u8(sf), want_sf)
    assert np.array_equal(host_u8(q), want_q)
