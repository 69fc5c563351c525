"""Argument blocks of a cache whose dimensions of size 1 lie at strides of their own, which reach nothing: on CPU, with tensors in host memory that nothing reads."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def test_dimensions_of_one(g):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    c = g.kv_cache(z(5, 2, 16, 64)[:1], z(1, 2, 16, 64))          # one page of a larger cache, and a page alone
    assert (c.pages, c.heads, c.head_stride, c.token_stride) == (1, 2, 16 * 64, 64)
    c = g.kv_cache(z(5, 1, 16, 64), z(5, 16, 1, 64).transpose(1, 2))  # one head: before the tokens or behind them
    assert (c.pages, c.heads, c.page_stride, c.token_stride) == (5, 1, 16 * 64, 64)
    for other in (z(2, 16, 64 + 8, 64)[:, :, :64].transpose(1, 2), z(2, 64, 16, 64)[:, :, :, :32]):
        with pytest.raises(ValueError, match="strides"):
            g.kv_cache(z(2, 64, 16, 64), other)
