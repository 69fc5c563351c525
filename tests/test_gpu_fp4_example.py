"""The example of an MLP block in 4 bits runs and stays near the same block in fp32.

An operand's relative error is about 0.1 (4-bit elements under group scales: a uniform error of a quarter to a half
step on two or three significant levels), a product of two of them 0.14 and a chain of two products 0.2 in the
direction of the block's output; a cosine of 1 / sqrt(1 + 0.2^2) = 0.98 follows, for the gradients that pass both
products and their own quantisation 1 / sqrt(1 + 0.35^2) = 0.94. The stream itself is dominated by the residual."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp4_mlp_block.py")


def test_block_in_4_bits():
    spec = importlib.util.spec_from_file_location("fp4_mlp_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    found = m.main()
    assert set(found) == {("NVFP4", 2048), ("NVFP4", 1), ("MXFP4", 2048), ("MXFP4", 1)}
    for case, cos in found.items():
        for k, v in cos.items():
            assert v > (0.98 if k in ("r", "h") else 0.9), (case, k, v)
