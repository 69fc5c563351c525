"""Pins of the 4-bit oracle: code values, the cast against a search in exact rationals, scale
rules, the byte layout, and the product on hand-made operands. No GPU."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp4, fp8

FMTS = [fp4.NV, fp4.MX]


def test_code_values_from_the_bit_fields():
    for c in range(16):
        e, f = (c >> 1) & 3, c & 1
        mag = f * 0.5 if e == 0 else (1 + f * 0.5) * 2.0 ** (e - 1)
        assert fp4.code_values(np.array([c]))[0] == (-mag if c & 8 else mag)


def test_cast_is_nearest_with_ties_to_even():
    grid = [Fraction(v) for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]
    points = np.unique(np.concatenate([np.linspace(-7, 7, 1121), np.float32(np.linspace(-7, 7, 997))]))
    for v in points:
        a = min(abs(Fraction(float(v))), Fraction(6))
        d = [abs(a - m) for m in grid]
        near = [i for i in range(8) if d[i] == min(d)]
        want = near[0] if len(near) == 1 else next(i for i in near if i % 2 == 0)
        got = int(fp4.cast_e2m1(np.array([v]))[0])
        assert got & 7 == want and (got >> 3) == int(v < 0 or (v == 0 and np.signbit(v))), v
    assert fp4.cast_e2m1(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, np.inf])).tolist() == [0, 2, 2, 4, 4, 6, 6, 7]


def test_mx_exponent_is_the_smallest_that_does_not_saturate():
    for a in [2.0 ** -130, 1e-30, 0.4, 3.0, 6.0, 6.03, 7.9, 12.0, 12.1, 448.0, fp4.BF16_MAX]:
        e = fp4.mx_exponent(a)
        assert 6 * 2.0 ** e >= a and (e == -127 or 6 * 2.0 ** (e - 1) < a)
    assert fp4.mx_exponent(0.0) == 0 and fp4.mx_exponent(2.0 ** -140) == -127


@pytest.mark.parametrize("fmt", FMTS)
def test_representable_values_come_back(fmt):
    rng = np.random.default_rng(fmt)
    g = fp4.GROUP[fmt]
    codes = rng.integers(0, 16, (5, 3 * g)).astype(np.uint8)
    codes[:, ::g] = 7  # each group holds its largest value, so its scale is recovered
    scale = np.repeat(np.array([[0.5, 2.0, 8.0]]), g, axis=1)
    x = fp4.code_values(codes) * scale
    q, b = fp4.quantize(x, fmt)
    assert np.array_equal(fp4.values(q, b, fmt), x)


def test_special_groups():
    for fmt in FMTS:
        g = fp4.GROUP[fmt]
        x = np.zeros((1, 4 * g), dtype=np.float32)
        x[0, 0] = np.nan
        x[0, g] = np.inf
        x[0, g + 1] = -1.0
        x[0, 3 * g] = -0.0
        q, b = fp4.quantize(x, fmt)
        assert b[0, 0] == fp4.NAN_SCALE[fmt] and not q[0, :g].any()
        assert q[0, g] == 7 and b[0, 1] == (0x7E if fmt == fp4.NV else 126 + 127)
        assert b[0, 2] == (0 if fmt == fp4.NV else 127) and not q[0, 2 * g:3 * g].any()
        assert q[0, 3 * g] == 8


def test_relative_error_of_a_group():
    # largest element within half a step (4 to 6) after the scale's own rounding (2^-4 of it, E4M3)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 96)).astype(np.float32)
    for fmt in FMTS:
        q, b = fp4.quantize(x, fmt)
        c = np.repeat(fp4.scale_value(b, fmt), fp4.GROUP[fmt], axis=1)
        v = fp4.values(q, b, fmt)
        assert (np.abs(v - x) <= c * 1.0 + (np.abs(x) / 16 if fmt == fp4.NV else 0)).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mn,k", [(1, 1), (3, 33), (128, 64), (129, 200), (300, 1024)])
def test_pack_and_unpack(fmt, mn, k):
    rng = np.random.default_rng(mn + k)
    codes = rng.integers(0, 16, (mn, k)).astype(np.uint8)
    byte = rng.integers(0, 255, (mn, -(-k // fp4.GROUP[fmt]))).astype(np.uint8)
    q, sf = fp4.pack(codes, byte, fmt)
    assert q.shape == (mn, fp4.row_bytes(k)) and sf.size == fp4.scale_bytes(fmt, mn, k) and sf.size % 512 == 0
    c2, b2 = fp4.unpack(q, sf, fmt, mn, k)
    assert np.array_equal(codes, c2) and np.array_equal(byte, b2)
    # the layout by its words: row m, group g
    m, g = mn - 1, byte.shape[1] - 1
    atom = (m // 128) * -(-byte.shape[1] // 4) + g // 4
    assert sf[atom * 512 + (m % 32) * 16 + ((m % 128) // 32) * 4 + g % 4] == byte[m, g]


def test_product_by_hand():
    a = fp4.values(np.array([[7, 2]], dtype=np.uint8), np.array([[0x38]], dtype=np.uint8), fp4.NV)  # 6, 1 at scale 1
    b = fp4.values(np.array([[1, 10]], dtype=np.uint8), np.array([[0x40]], dtype=np.uint8), fp4.NV)  # .5, -1 at scale 2
    c, mag = fp4.scaled_mm(a, b, 2.0, 3.0)
    assert c[0, 0] == (6 * 1.0 - 1 * 2.0) * 6 and mag[0, 0] == 8 * 6
    assert fp8.decode(0x38, fp8.E4M3) == 1.0 and fp8.decode(0x40, fp8.E4M3) == 2.0
