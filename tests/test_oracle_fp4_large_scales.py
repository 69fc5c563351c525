"""The oracle's NVFP4 under tensor scales so large that s / c would overflow: every factor is finite, zeros stay zeros, and a
code under its raised scale is the nearest one to its element."""
import numpy as np
import pytest

from oracle import fp4, fp8


@pytest.mark.parametrize("s", [2.0 ** 118, np.nextafter(np.float32(2.0 ** 119), np.float32(0)), 1e36, 3e37, 3.4e38])
def test_codes_stand_for_their_elements(s):
    s = np.float32(s)
    rng = np.random.default_rng(int(np.log2(s)))
    x = (rng.uniform(-1, 1, (400, 32)) * np.exp2(-rng.uniform(0, 18, (400, 1))) * 2688 / np.float64(s)).astype(np.float32)
    x[:, 3], x[:, 20], x[5] = 0.0, -0.0, 0.0
    with np.errstate(over="raise", invalid="raise"):
        codes, byte = fp4.quantize(x, fp4.NV, s)
    assert ((codes & 7)[:, [3, 20]] == 0).all() and (byte[5] == 0).all()
    c = np.repeat(fp4.scale_value(byte, fp4.NV), 16, axis=1)
    least = float(fp8.decode_array(np.array([fp4.least_scale(s)], dtype=np.uint8), fp8.E4M3)[0])
    assert ((c == 0) | (c >= least)).all()
    with np.errstate(over="ignore"):
        assert np.isfinite(s / np.float32(least)) and (fp4.least_scale(s) == 1 or not np.isfinite(s / np.float32(fp8.decode_array(
            np.array([fp4.least_scale(s) - 1], dtype=np.uint8), fp8.E4M3)[0])))
    live = c > 0
    v = np.float64(x) * np.float64(s)
    z = v / np.where(live, c, 1.0)
    # two fp32 roundings, of s / c and of the product, each within 2^-24
    low, high = (fp4.code_values(fp4.cast_e2m1(z * (1 + e))) for e in (-(2.0 ** -22), 2.0 ** -22))
    got = fp4.code_values(codes)
    assert ((got >= np.minimum(low, high)) & (got <= np.maximum(low, high)))[live].all()
    assert (np.abs(v)[~live] <= 6 * 2.0 ** -10 * 1.001).all()


def test_scales_up_to_2_to_the_118_are_as_they_were():
    assert fp4.least_scale(np.float32(1)) == 1 and fp4.least_scale(np.float32(2.0 ** 118)) == 1
