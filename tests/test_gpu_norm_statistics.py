"""The statistics that the norms' forward stores, both of them, in every kernel: against the oracle, in buffers that held something
else before.

Bound: a row's sums are within e = (D / 512 + 16) 2^-24 of themselves. r' carries 2 e of the magnitudes a of its terms (its
norm's statistic and a few roundings), and the subtracted mean as much of theirs; so the mean is off by at most 4 e mean(a)
(twice that taken), and 1 / root by e and, as the root is a length, by the length of the elements' errors over the root:
4 e sqrt(mean(a^2)) / root (twice both taken for the terms of second order)."""
import numpy as np
import pytest
import torch

import test_gpu_block_norm as bn
from test_gpu_block_norm import Case, rel_stat, terms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def statistics(c):
    """(stat_post, stat_pre) as the forward stores them over a sentinel; they are the last rows of longer buffers."""
    whole = [torch.full((c.T + 2, 2), 777.0, device="cuda") for _ in range(2)]
    post, pre = (w[1:-1] for w in whole)
    f = c.plan(r_out=c.out(c.stream), h=c.out(c.block), stat_post=post, stat_pre=pre)
    c.g.fp8_block_norm_fwd(f)
    torch.cuda.synchronize()
    assert all((w[0] == 777.0).all() and (w[-1] == 777.0).all() for w in whole)
    return post.double().cpu().numpy(), pre.double().cpu().numpy()


def check(c):
    post, pre = statistics(c)
    e, (a, _) = rel_stat(c), terms(c)
    for got, kind, want, mag, carried in ((post, c.post, c.ref["post"], np.abs(c.vo) if c.vo is not None else np.zeros((c.T, c.D)), 0), (pre, c.pre, c.ref["pre"], a, 1)):
        mean, inv = want
        if kind == 2:
            assert (np.abs(got[:, :1] - mean) <= (8 * e if carried else e) * mag.mean(axis=1, keepdims=True)).all()
        else:
            assert (got[:, 0] == 0).all()
        if kind == 0:
            assert (got[:, 1] == 1).all()
        else:
            rel = 2 * (e + 4 * e * np.sqrt((mag ** 2).mean(axis=1, keepdims=True)) * inv)
            assert (np.abs(got[:, 1:] / inv - 1) <= rel).all(), (np.abs(got[:, 1:] / inv - 1) / rel).max()


@pytest.mark.parametrize("T,D", [(1, 1), (3, 40), (5, 1537), (40, 256), (33, 2048), (9, 8192), (3, 16384), (2, 20000), (3, 8195)])
@pytest.mark.parametrize("post,pre", [(1, 2), (2, 1), (0, 1), (2, 0), (0, 2)])
def test_few_rows(g, T, D, post, pre):
    for stream, block in (("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")):
        check(Case(g, T, D, stream, block, post, pre, rows=2))


def test_without_a_block(g):
    for D in (96, 131, 4096):
        check(Case(g, 7, D, o=False, pre=2))


@pytest.mark.parametrize("D", [768, 1024, 1032, 3000, 4096, 5120, 6152, 8192])
@pytest.mark.parametrize("post,pre", [(1, 2), (2, 1), (0, 1), (2, 0)])
def test_rows_ahead(g, D, post, pre):
    """Enough rows for the kernel that keeps rows ahead in shared memory."""
    per = 32 if D < 1024 else 8 if D <= 4096 else 4
    T = per * torch.cuda.get_device_properties(0).multi_processor_count + 5
    check(Case(g, T, D, "bf16", "bf16", post, pre, rows=100))
    if post == 1:
        check(Case(g, T, D, "f32", "f32" if D % 8 == 0 else "bf16", post, pre, rows=0))
