"""Microscaled 4-bit operands (oracle; test infrastructure): the E2M1 cast, group scales, the
byte layout of codes and scales, and the product, in numpy.

E2M1: sign, 2 exponent bits (bias 1), 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
NVFP4: c = e4m3(fl32(fl32(a s) / 6)) per 16 elements (a: the group's amax, s the tensor's scale), a c that is
       not 0 raised to the smallest one whose fl32(s / c) is finite,
       code = e2m1(fl32(x fl32(s / c))); the fp32 roundings are part of the definition.
MXFP4: 2^e per 32 elements, e the smallest integer with 6 2^e >= a (0 for a = 0, at least -127).
A NaN in a group: scale NaN, zero codes. An infinity counts as the largest finite bf16 in a.

The pages stop at 8 bits; the readings above are this library's (parity unpinned).
Pins: tests/test_oracle_fp4.py.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8

NV, MX = 0, 1
GROUP = {NV: 16, MX: 32}
FILL = {NV: 0, MX: 127}
NAN_SCALE = {NV: 0x7F, MX: 0xFF}
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BF16_MAX = float(np.float64(2.0) ** 127 * (2 - 2.0 ** -7))


def cast_e2m1(v) -> np.ndarray:
    """Nearest of the 8 magnitudes, ties to the even code, saturating; sign (of zero too) kept."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    best = np.zeros(v.shape, dtype=np.uint8)
    dist = np.full(v.shape, np.inf)
    for code, m in enumerate(VALUES):
        d = np.abs(a - m)
        take = (d < dist) | ((d == dist) & (code % 2 == 0))
        best = np.where(take, code, best).astype(np.uint8)
        dist = np.where(take, d, dist)
    return best | np.where(np.signbit(v), 8, 0).astype(np.uint8)


def code_values(codes) -> np.ndarray:
    codes = np.asarray(codes)
    return np.where(codes & 8, -1.0, 1.0) * VALUES[codes & 7]


def mx_exponent(a: float) -> int:
    if a == 0:
        return 0
    m, e = math.frexp(a)  # a = m 2^e, 0.5 <= m < 1
    return max(-127, e - 3 if m <= 0.75 else e - 2)


def least_scale(s) -> int:
    """The smallest E4M3 code above 0 under which the tensor scale s (finite, above 0) gives a finite factor."""
    with np.errstate(over="ignore"):
        finite = np.isfinite(np.float32(s) / fp8.decode_array(np.arange(1, 127, dtype=np.uint8), fp8.E4M3).astype(np.float32))
    return 1 + int(np.argmax(finite))


def scale_value(byte, fmt) -> np.ndarray:
    byte = np.asarray(byte, dtype=np.uint8)
    if fmt == NV:
        return fp8.decode_array(byte, fp8.E4M3)
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))


def quantize(x, fmt, s=np.float32(1.0)):
    """x [MN, K] (fp32 or bf16 values) -> codes [MN, K] uint8 and scale bytes [MN, groups] uint8."""
    x = np.asarray(x, dtype=np.float32)
    mn, k = x.shape
    g = GROUP[fmt]
    n = -(-k // g)
    z = np.zeros((mn, n * g), dtype=np.float32)
    z[:, :k] = x
    z = z.reshape(mn, n, g)
    nan = np.isnan(z).any(axis=2)
    with np.errstate(all="ignore"):
        a = np.abs(np.where(np.isnan(z), 0, z)).max(axis=2).astype(np.float32)
        if fmt == NV:
            a = np.where(np.isinf(a), np.float32(BF16_MAX), a)
            t = (a * np.float32(s)).astype(np.float32) / np.float32(6.0)
            byte = fp8.cast(t, fp8.E4M3)
            byte = np.where(byte > 0, np.maximum(byte, least_scale(s)), 0).astype(np.uint8)
            c = fp8.decode_array(byte, fp8.E4M3).astype(np.float32)
            mul = np.where(c > 0, np.float32(s) / np.where(c > 0, c, np.float32(1)), np.float32(0)).astype(np.float32)
        else:
            e = np.array([mx_exponent(min(float(v), BF16_MAX)) for v in a.reshape(-1)]).reshape(a.shape)
            byte = (e + 127).astype(np.uint8)
            mul = np.ldexp(np.float32(1.0), -e).astype(np.float32)
        codes = cast_e2m1((z * mul[:, :, None]).astype(np.float32))
    codes = np.where(nan[:, :, None], 0, codes).astype(np.uint8)
    byte = np.where(nan, NAN_SCALE[fmt], byte).astype(np.uint8)
    return codes.reshape(mn, -1)[:, :k], byte


def values(codes, byte, fmt) -> np.ndarray:
    """float64 values of codes [MN, K] under their group scales (no tensor scale)."""
    k = np.asarray(codes).shape[1]
    return code_values(codes) * np.repeat(scale_value(byte, fmt), GROUP[fmt], axis=1)[:, :k]


def row_bytes(k: int) -> int:
    return -(-k // 32) * 16


def scale_bytes(fmt, mn: int, k: int) -> int:
    groups = -(-k // GROUP[fmt])
    return -(-mn // 128) * -(-groups // 4) * 512


def scale_offsets(fmt, mn: int, k: int) -> np.ndarray:
    """Byte of (row, group) in the scale atoms, [MN, groups]."""
    groups = -(-k // GROUP[fmt])
    m, g = np.arange(mn)[:, None], np.arange(groups)[None, :]
    return ((m // 128) * -(-groups // 4) + g // 4) * 512 + 16 * (m % 32) + 4 * ((m // 32) % 4) + g % 4


def pack(codes, byte, fmt):
    """The library's bytes: codes [MN, row_bytes] and the scale atoms, padding included."""
    mn, k = codes.shape
    full = np.zeros((mn, 2 * row_bytes(k)), dtype=np.uint8)
    full[:, :k] = codes
    sf = np.full(scale_bytes(fmt, mn, k), FILL[fmt], dtype=np.uint8)
    sf[scale_offsets(fmt, mn, k)] = byte
    return full[:, 0::2] | (full[:, 1::2] << 4), sf


def unpack(q, sf, fmt, mn: int, k: int):
    q = np.asarray(q, dtype=np.uint8).reshape(mn, row_bytes(k))
    codes = np.empty((mn, 2 * q.shape[1]), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = q & 15, q >> 4
    return codes[:, :k], np.asarray(sf, dtype=np.uint8)[scale_offsets(fmt, mn, k)]


def scaled_mm(va, vb, d_a=1.0, d_b=1.0):
    """(C, magnitude sum): C = d_a d_b va vb^T in fp64 of operand values [M, K], [N, K], with
    d_a d_b rounded to fp32 as the library multiplies them; Sum |a b| alongside for error bounds."""
    d = float(np.float32(np.float32(d_a) * np.float32(d_b)))
    return va @ vb.T * d, np.abs(va) @ np.abs(vb).T * abs(d)
