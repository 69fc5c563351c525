"""The oracle of the heads' operators: gradients against differences, the rotation against complex numbers, the 8-bit form against a search
through all codes, attention against a direct sum; and the library's frequencies, made on the host, against the oracle's."""
import math

import numpy as np
import pytest

from oracle import heads


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, theta = rng.standard_normal((3, 2, 10)), rng.standard_normal((3, 4))
    y = heads.rotate(x, theta, interleaved, 1.5)
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    z = (a + 1j * b) * 1.5 * np.exp(1j * theta)[:, None]
    got = (y[..., 0:8:2], y[..., 1:8:2]) if interleaved else (y[..., :4], y[..., 4:8])
    assert np.allclose(got[0], z.real) and np.allclose(got[1], z.imag) and np.array_equal(y[..., 8:], x[..., 8:])


@pytest.mark.parametrize("normed", [False, True])
def test_gradients_against_differences(normed):
    rng = np.random.default_rng(2)
    x, w, theta = rng.standard_normal((2, 3, 8)), 1 + 0.1 * rng.standard_normal(8), rng.standard_normal((2, 3))
    dy = rng.standard_normal(x.shape)
    f = lambda x, w: (heads.forward(x, w, 1e-3, theta, False, 0.9, normed) * dy).sum()  # noqa: E731
    dx, dw = heads.backward(dy, x, w, 1e-3, theta, False, 0.9, normed)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if normed:
        for i in range(8):
            e = np.zeros(8)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_angles_are_exact_far_out():
    f = [1 << 63, 1, (1 << 64) - 1, 0x123456789ABCDEF]
    a = heads.angle([0, 1, 3, (1 << 31) - 1, -5], f)
    assert a[0].tolist() == [0, 0, 0, 0] and a[2, 0] == pytest.approx(math.pi) and a[3, 0] == pytest.approx(math.pi)
    assert a[3, 1] == (2 ** 31 - 1) * 2 * math.pi / 2 ** 64


def test_eight_bit_groups():
    v = heads.e4m3_values()
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and np.isnan(v[0x7F]) and v[0xFE] == -448
    x = np.zeros((7, 32))
    x[1, 3], x[2, 3], x[3, 3], x[4, 3], x[5, 3], x[6, 3] = 448, 448.0001, 449 * 2.0 ** -140, np.inf, np.nan, 224
    assert heads.mx_exponents(x)[:, 0].tolist() == [0, 0, 1, -127, 120, 128, -1]


def test_attention_against_a_direct_sum():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 1, 8, 4)), rng.standard_normal((2, 1, 8, 4))
    q = rng.standard_normal((2, 2, 4))
    out, lse, _, _ = heads.attention(q, k, v, [0, 2], [10], np.array([[1, 0]]), 0.5, window=9)
    keys, vals = np.concatenate([k[1, 0], k[0, 0]]), np.concatenate([v[1, 0], v[0, 0]])
    for t, (a, b) in enumerate(((0, 9), (1, 10))):
        e = np.exp(0.5 * keys[a:b] @ q[t, 1])
        assert np.allclose(out[t, 1], e @ vals[a:b] / e.sum()) and np.isclose(lse[t, 1], np.log(e.sum()))
    out, lse, _, _ = heads.attention(q, k, v, [0, 2], [1], np.array([[1, 0]]), 0.5)
    assert np.array_equal(out[0], np.zeros((2, 4))) and np.all(lse[0] == -np.inf) and np.allclose(out[1], vals[0])


@pytest.mark.parametrize("rot", [2, 4, 32, 96, 128, 256])
@pytest.mark.parametrize("kind", ["plain", "linear", "base", "parts", "by_index"])
def test_frequencies(g, rot, kind):
    import ctypes
    if kind == "base" and rot < 4:
        pytest.skip("a stretched base needs four dimensions")
    code = {"plain": g.FP8_ROPE_PLAIN, "linear": g.FP8_ROPE_LINEAR, "base": g.FP8_ROPE_BASE, "parts": g.FP8_ROPE_PARTS, "by_index": g.FP8_ROPE_PARTS_BY_INDEX}[kind]
    for base, factor, original, low, high in ((10000.0, 8.0, 8192.0, 1.0, 4.0), (500000.0, 2.5, 4096.0, 1.0, 32.0), (1.5, 0.5, 100.0, 0.01, 0.5)):
        t = (ctypes.c_uint64 * (rot // 2))()
        g.fp8_rope_turns(rot, base, code, factor, original, low, high, t)
        want = heads.turns(rot, base, kind, factor, original, low, high)
        # 64 fractional bits, of a number computed in 53
        got = np.array([int(x) for x in t], dtype=np.float64) / 2.0 ** 64
        assert np.all(np.abs(got - want % 1.0) <= 2.0 ** -46 * want + 2.0 ** -64)


def test_frequencies_refused(g):
    import ctypes
    t = (ctypes.c_uint64 * 128)()
    inv, un = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_UNSUPPORTED
    for status, args in ((inv, (3, 1e4, 0, 1, 0, 1, 4)), (inv, (-2, 1e4, 0, 1, 0, 1, 4)), (un, (258, 1e4, 0, 1, 0, 1, 4)), (inv, (64, 1e4, 5, 1, 0, 1, 4)),
                         (inv, (64, 1.0, 0, 1, 0, 1, 4)), (inv, (64, math.inf, 0, 1, 0, 1, 4)), (inv, (64, math.nan, 0, 1, 0, 1, 4)), (inv, (64, 1e4, 1, 0.0, 0, 1, 4)),
                         (inv, (2, 1e4, 2, 2.0, 0, 1, 4)), (inv, (64, 1e4, 3, 8.0, 0.0, 1, 4)), (inv, (64, 1e4, 3, 8.0, 8192.0, 4, 4)), (inv, (64, 1e4, 4, 8.0, 8192.0, 0, 4))):
        with pytest.raises(g.Fp8Error) as e:
            g.fp8_rope_turns(*args, t)
        assert e.value.status == status, args
    with pytest.raises(g.Fp8Error):
        g.fp8_rope_turns(64, 1e4, 0, 1, 0, 1, 4, None)
    assert g.fp8_rope_turns(0, 1e4, 0, 1, 0, 1, 4, None) == 0
    assert g.rope_turns(8, 1e4, device="cpu").tolist()[0] == int(2 ** 64 / (2 * math.pi))  # (as near as 53 bits come)
