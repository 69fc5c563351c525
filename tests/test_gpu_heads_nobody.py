"""Rows of nobody, before the first sequence and behind the last one: whatever they hold, no other row's result and no place of the cache
changes by a bit, and they are not written."""
import pytest
import torch

from test_gpu_kv_append import Batch
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def beginnings(b):
    """The sequences from row 2 on."""
    b.q_start = b.q_start + 2
    return [0, 1] + list(range(int(b.q_start[-1]), b.T))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("off, rot, norm", [(0, 64, True), (1, 64, True), (0, 32, False), (3, 20, False)])
def test_append(g, mx, off, rot, norm):
    results = []
    for value in (None, float("nan"), float("inf")):
        b = Batch(g, [5, 1, 9], [17, 40, 9], 3, 2, 64, 16, mx, False, extra=9, off=off)
        nobody = beginnings(b)
        if value is not None:
            b.x[nobody] = value
        f = g.qk_rope(b.T, 3, 2, 64, rot, 0, norm=int(norm), turns=g.rope_turns(rot, 1e4), q=b.q, k=b.k, v=b.v, q_out=b.q_out)
        g.fp8_kv_append(f, b.kv(g), b.batch(g))
        assert torch.all(b.q_out[nobody] == 5.0)
        results.append([b.q_out, *b.cache] + (b.units if mx else []))
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("new, total, heads_", [([1, 1, 1], [100, 700, 33], (8, 2)), ([40, 3], [300, 900], (4, 2)), ([130, 5], [400, 90], (6, 2)), ([1], [9000], (4, 1))], ids=str)
def test_attention(g, mx, new, total, heads_):
    results = []
    for value in (None, float("nan"), float("inf")):
        c = Case(g, new, total, *heads_, 128, 16, mx, extra=200)
        nobody = beginnings(c)
        if value is not None:
            c.q[nobody] = value
        c.run()
        assert torch.all(c.out[nobody] == 9.0) and torch.all(c.lse[nobody] == 9.0)
        results.append((c.out, c.lse))
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))
