"""NVFP4 under tensor scales so large that a group's factor s / c would overflow: the group's scale is raised until it does
not, so zeros stay zero codes and the codes stand for their elements. Bit for bit against the oracle, all ways."""
import numpy as np
import pytest
import torch

from datagen import bf16_bits_from_f32, f32_from_bf16_bits
from oracle import fp4

from gpu_util import host_u8
from test_gpu_fp4_quant import check, quantize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def small(seed, rows, cols, amax):
    """Groups of every size down to the subnormals, zeros of both signs among them."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(-1, 1, (rows, cols)) * np.exp2(-rng.uniform(0, 16, (rows, 1)))
    x[rng.random((rows, cols)) < 0.3] = 0.0
    x[rng.random((rows, cols)) < 0.1] = -0.0
    x[0, 0] = 1.0
    return f32_from_bf16_bits(bf16_bits_from_f32((x * amax).astype(np.float32)))


@pytest.mark.parametrize("amax", [1e-32, 2e-33, 1e-34, 1e-35, 8e-36])
@pytest.mark.parametrize("which", ["rows", "cols", "both"])
@pytest.mark.parametrize("rows,cols", [(40, 72), (130, 264), (33, 37)])
def test_quantize(g, amax, which, rows, cols):
    x = small(rows + cols, rows, cols, amax)
    st = g.TensorState(16)
    out = quantize(g, x, fp4.NV, which, st)
    s = np.float32(2688) / np.abs(x).max()
    assert st.snapshot()["scale"] == s
    check(out, x, fp4.NV, s)


@pytest.mark.parametrize("T,D", [(3, 64), (40, 256), (1300, 1056), (2, 16416)])
@pytest.mark.parametrize("scale", [2.0 ** 119, 1e37, 3e38])
def test_norm_into_4_bits(g, T, D, scale):
    """h of the norm against its own fp32 output."""
    gen = torch.Generator("cuda").manual_seed(T + D)
    r = torch.randn(T, D, generator=gen, device="cuda") * torch.exp2(-16 * torch.rand(T, D // 32, 1, generator=gen, device="cuda")).expand(T, D // 32, 32).reshape(T, D)
    r[torch.rand(T, D, generator=gen, device="cuda") < 0.3] = 0.0
    o = torch.zeros(T, D, device="cuda")
    w = torch.full((D,), 700.0 / scale, device="cuda")
    q = torch.full((T, g.fp4_row_bytes(D)), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((g.fp4_scale_bytes(fp4.NV, T, D),), 0xA5, dtype=torch.uint8, device="cuda")
    h = torch.empty(T, D, device="cuda")
    f = g.block_norm(T, D, g.FP8_DT_F32, g.FP8_DT_F32, pre=g.FP8_NORM_RMS, r=r, o=o, w_pre=w, h=h, hq=q, hsf=sf, h_fmt=fp4.NV,
                     h_scale=torch.tensor([scale], device="cuda"))
    g.fp8_block_norm_fwd(f)
    torch.cuda.synchronize()
    want_q, want_sf = fp4.pack(*fp4.quantize(h.cpu().numpy(), fp4.NV, np.float32(scale)), fp4.NV)
    assert np.array_equal(host_u8(sf), want_sf)
    assert np.array_equal(host_u8(q), want_q)
