"""The forward of the norms on both sides of the number of rows from which rows are kept ahead in shared memory (per SM: 4 above 4096
columns, 8 from 1024 on, 32 below), made from the device's number of SMs; into 4 bits at every width of a team; offsets
past 32 bits there."""
import pytest
import torch

import test_gpu_block_norm as bn
import test_gpu_long_offsets as far
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def threshold(D):
    return (4 if D > 4096 else 8 if D >= 1024 else 32) * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("D", [520, 1016, 1024, 4096, 4104, 6144, 6152, 8192])
@pytest.mark.parametrize("past", [-1, 0, 1, 100])
@pytest.mark.parametrize("stream,block", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_forward(g, D, past, stream, block):
    c = bn.Case(g, threshold(D) + past, D, stream, block, 1 + past % 2, 2 - past % 2, 100)
    c.forward()
    bn.check_forward(c)


# teams of 1 to 8, 9 to 12 and 13 to 16 warps, whole and ragged
@pytest.mark.parametrize("D", [544, 1024, 2080, 4096, 4128, 6144, 6176, 7200, 8192])
@pytest.mark.parametrize("fmt", [fp4.NV, fp4.MX])
def test_into_4_bits(g, fmt, D):
    for T in (threshold(D) - 3, threshold(D) + 3):
        bn.test_forward_into_4_bits(g, fmt, T, D, "bf16", "bf16")


@pytest.mark.parametrize("fmt", [fp4.NV, fp4.MX])
def test_into_4_bits_from_fp32(g, fmt):
    for D in (2048, 6176, 8192):
        bn.test_forward_into_4_bits(g, fmt, threshold(D) + 3, D, "f32", "f32")


@pytest.mark.parametrize("D,stream", [(768, torch.bfloat16), (1024, torch.float32), (4104, torch.bfloat16)])
def test_offsets_past_32_bits(g, D, stream):
    far.test_norms(g, D, stream, far.PITCH)
