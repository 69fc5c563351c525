"""Batches whose beginnings fall: unused entries of zeros behind the last sequence, a step back between two sequences. Append and attention
take the same rows for the same sequences, those that the oracle names (bounds: as in the operators' own tests)."""
import numpy as np
import pytest
import torch

from oracle import heads
from test_gpu_kv_append import Batch, check
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


STARTS = {  # beginnings of sequences of which those that have rows hold them alone
    "zeros behind": lambda n, unused: [3 * i for i in range(n + 1)] + [0] * unused,
    "negative behind": lambda n, unused: [3 * i for i in range(n + 1)] + [-7] * unused,
    "from the end": lambda n, unused: [3 * i for i in range(n + 1)] + [1 << 20] + [0] * (unused - 1) if unused else [3 * i for i in range(n + 1)],
    "one step back": lambda n, unused: [3 * (n // 2) + 3 * i for i in range(n - n // 2 + 1)] + [0] * (unused + 1) + [3 * i for i in range(1, n // 2 + 1)],
}


@pytest.mark.parametrize("kind", STARTS)
@pytest.mark.parametrize("n, unused", [(1, 1), (2, 0), (5, 3), (5, 59), (40, 24), (40, 1000), (200, 70)])
def test_beginnings_that_fall(g, kind, n, unused):
    start = STARTS[kind](n, unused)
    seqs = len(start) - 1
    held = [max(0, min(b, 3 * n + 2) - max(0, a)) for a, b in zip(start, start[1:])]  # (rows are 3 n and two of nobody)
    assert sum(held) <= 3 * n + 2
    total = [5 + 3 * (i % 7) if h else 9 for i, h in enumerate(held)]
    b = Batch(g, [3] * seqs, total, 4, 2, 64, 16, False, False, extra=3 * n + 2 - 3 * seqs)
    b.q_start = np.array(start, dtype=np.int32)
    check(g, b, 64, False)
    c = Case(g, [3] * seqs, total, 4, 2, 64, 16, extra=3 * n + 2 - 3 * seqs)
    c.q_start = np.array(start, dtype=np.int32)
    c.run()
    c.check()
    assert sum(s >= 0 for s, _ in heads.places(start, total, 3 * n + 2)) == sum(held)
