"""The product of 4-bit operands on the GPU against the oracle.

Exact cases: codes and scales whose products and sums fit fp32 exactly, with a different scale for
every row and group, so a scale byte, a row or a code read from the wrong place changes a result.
Random cases: within a bound. fp32 accumulation over K in steps of 64 adds at most a relative 2^-22
of the magnitude sum per step (the tensor cores may truncate), and 2^-22 inside a step's sum of
products; then one rounding to the output type."""
import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

FMTS = [fp4.NV, fp4.MX]


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def operand(rng, fmt, mn, k, exact):
    groups = -(-k // fp4.GROUP[fmt])
    if exact:  # values 0, +-1, +-2, +-3 under scales 1, 2, 4: sums of K <= 2^14 stay below 2^24
        codes = rng.choice(np.array([0, 2, 4, 5, 10, 12, 13], dtype=np.uint8), (mn, k))
        e = rng.integers(0, 3, (mn, groups))
        byte = (0x38 + 8 * e if fmt == fp4.NV else 127 + e).astype(np.uint8)
    else:
        codes = rng.integers(0, 16, (mn, k)).astype(np.uint8)
        byte = rng.integers(0x20, 0x50, (mn, groups)).astype(np.uint8) if fmt == fp4.NV else rng.integers(120, 132, (mn, groups)).astype(np.uint8)
    q, sf = fp4.pack(codes, byte, fmt)
    return torch.from_numpy(q).cuda(), torch.from_numpy(sf).cuda(), fp4.values(codes, byte, fmt)


def product(g, a, b, m, n, k, fmt, f32, da=None, db=None, pad=0, stream=None):
    """C as float64 [m, n]; what lies past its columns and rows must stay as it was."""
    ld = -(-n // 8) * 8 + pad
    c = torch.full((m + 1, ld), 3.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g.fp4_scaled_mm(a[0], a[1], b[0], b[1], m, n, k, fmt, da, db, c, g.FP8_DT_F32 if f32 else g.FP8_DT_BF16, ld, stream)
    torch.cuda.synchronize()
    g.fp8_poll_device_error()
    h = c.float().cpu().numpy().astype(np.float64)
    assert (h[:, n:] == 3.0).all() and (h[m:] == 3.0).all()
    return h[:m, :n]


def to_bf16(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).float().numpy().astype(np.float64)


# tokens from one to several tiles, K inside a group, an atom, a tile and past several tiles, N ragged
SHAPES = [(1, 8, 16), (1, 1, 1), (1, 129, 33), (2, 256, 256), (7, 100, 1000), (16, 512, 4096), (17, 40, 300), (33, 1000, 520), (64, 128, 64),
          (65, 200, 96), (128, 128, 256), (129, 257, 511), (200, 136, 2048), (256, 256, 512), (300, 520, 1100), (513, 264, 128), (640, 1100, 260),
          (1, 4100, 8192), (48, 72, 16000), (700, 24, 9000)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact(g, fmt, m, n, k):
    rng = np.random.default_rng(m * 31 + n * 7 + k + fmt)
    a, b = operand(rng, fmt, m, k, True), operand(rng, fmt, n, k, True)
    want, _ = fp4.scaled_mm(a[2], b[2])
    assert np.abs(want).max() < 2 ** 24
    assert np.array_equal(product(g, a, b, m, n, k, fmt, True), want)
    assert np.array_equal(product(g, a, b, m, n, k, fmt, False), to_bf16(want))


@pytest.mark.parametrize("n", [2561, 2564, 2568, 2815, 2816])
@pytest.mark.parametrize("m", [2049, 2304])
@pytest.mark.parametrize("f32", [False, True])
def test_exact_many_tiles(g, m, n, f32):
    """Enough 256 x 256 tiles for every pair of SMs to take several, rows ending inside 16 bytes of the output."""
    k = 300
    rng = np.random.default_rng(m + n)
    a, b = operand(rng, fp4.NV, m, k, True), operand(rng, fp4.NV, n, k, True)
    want, _ = fp4.scaled_mm(a[2], b[2])
    assert np.array_equal(product(g, a, b, m, n, k, fp4.NV, f32), want if f32 else to_bf16(want))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 768, 3000), (20, 520, 1536), (130, 300, 777), (520, 1030, 2050), (1500, 640, 512)])
def test_random_within_the_bound(g, fmt, f32, m, n, k):
    rng = np.random.default_rng(m + n + k)
    a, b = operand(rng, fmt, m, k, False), operand(rng, fmt, n, k, False)
    da, db = torch.tensor([0.37], device="cuda"), torch.tensor([1.9], device="cuda")
    want, mag = fp4.scaled_mm(a[2], b[2], np.float32(0.37), np.float32(1.9))
    got = product(g, a, b, m, n, k, fmt, f32, da, db, pad=8)
    bound = (k / 64 + 2) * 2.0 ** -22 * mag + np.abs(want) * (2.0 ** -22 if f32 else 2.0 ** -8)
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()


@pytest.mark.parametrize("m,n,k", [(3, 300, 640), (300, 300, 640)])
def test_one_tensor_scale(g, m, n, k):
    rng = np.random.default_rng(1)
    a, b = operand(rng, fp4.NV, m, k, True), operand(rng, fp4.NV, n, k, True)
    want, _ = fp4.scaled_mm(a[2], b[2], 0.5)
    d = torch.tensor([0.5], device="cuda")
    assert np.array_equal(product(g, a, b, m, n, k, fp4.NV, True, d, None), want)
    assert np.array_equal(product(g, a, b, m, n, k, fp4.NV, True, None, d), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [5, 300])
def test_nan_scales_stay_in_their_rows(g, fmt, m):
    n, k = 200, 700
    rng = np.random.default_rng(2)
    a, b = operand(rng, fmt, m, k, True), operand(rng, fmt, n, k, True)
    want, _ = fp4.scaled_mm(a[2], b[2])
    sa, sb = a[1].clone(), b[1].clone()
    sa[int(fp4.scale_offsets(fmt, m, k)[3, -1])] = fp4.NAN_SCALE[fmt]
    sb[int(fp4.scale_offsets(fmt, n, k)[150, 0])] = fp4.NAN_SCALE[fmt]
    got = product(g, (a[0], sa), (b[0], sb), m, n, k, fmt, True)
    nan = np.zeros((m, n), bool)
    nan[3], nan[:, 150] = True, True
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], want[~nan])


def test_signed_largest_values(g):
    """Every code and scale at its largest: 448 * 6 on both sides, sums of one sign and of both."""
    m, n, k = 130, 140, 128
    for fmt, top in ((fp4.NV, 0x7E), (fp4.MX, 127 + 30)):
        codes = np.full((m, k), 7, np.uint8)
        cb = np.where(np.arange(n)[:, None] % 2, 15, 7).astype(np.uint8) * np.ones((1, k), np.uint8)
        ba, bb = np.full((m, -(-k // fp4.GROUP[fmt])), top, np.uint8), np.full((n, -(-k // fp4.GROUP[fmt])), top, np.uint8)
        qa, sa = fp4.pack(codes, ba, fmt)
        qb, sb = fp4.pack(cb, bb, fmt)
        t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        want, _ = fp4.scaled_mm(fp4.values(codes, ba, fmt), fp4.values(cb, bb, fmt))
        got = product(g, (t(qa), t(sa)), (t(qb), t(sb)), m, n, k, fmt, True)
        assert (np.abs(got - want) <= 2.0 ** -20 * np.abs(want)).all()


def test_empty_and_no_contraction(g):
    c = torch.full((4, 16), 5.0, device="cuda")
    g.fp4_scaled_mm(None, None, None, None, 3, 10, 0, fp4.NV, None, None, c, g.FP8_DT_F32, 16)
    g.fp4_scaled_mm(None, None, None, None, 0, 10, 64, fp4.NV, None, None, None, g.FP8_DT_F32, 16)
    torch.cuda.synchronize()
    h = c.cpu().numpy()
    assert (h[:3, :10] == 0).all() and (h[3:] == 5).all() and (h[:, 10:] == 5).all()


@pytest.mark.parametrize("m,n,k", [(4, 2048, 4096), (256, 128, 8192), (1024, 1024, 1024)])
def test_same_bits_every_time_and_on_another_stream(g, m, n, k):
    rng = np.random.default_rng(4)
    a, b = operand(rng, fp4.NV, m, k, False), operand(rng, fp4.NV, n, k, False)
    first = product(g, a, b, m, n, k, fp4.NV, True)
    s = torch.cuda.Stream()
    for i in range(4):
        assert np.array_equal(product(g, a, b, m, n, k, fp4.NV, True, stream=s if i % 2 else None), first)


def test_quantised_linear_layer_and_its_gradients(g):
    """Forward and both gradients of y = x W from quantised operands, against the same products of the
    oracle's quantised values (the operands' bits are tested elsewhere)."""
    from datagen import bf16_bits_from_f32, f32_from_bf16_bits
    from gpu_util import dev_bf16
    M, K, N = 200, 160, 272
    rng = np.random.default_rng(8)
    mk = lambda *s: f32_from_bf16_bits(bf16_bits_from_f32(rng.standard_normal(s).astype(np.float32)))  # noqa: E731
    x, w, dy = mk(M, K), mk(K, N), mk(M, N)
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731

    def both(v):
        r, c = v.shape
        b = [u8(r * g.fp4_row_bytes(c)), u8(g.fp4_scale_bytes(fp4.NV, r, c)), u8(c * g.fp4_row_bytes(r)), u8(g.fp4_scale_bytes(fp4.NV, c, r))]
        g.fp4_quantize(dev_bf16(bf16_bits_from_f32(v)), r, c, c, fp4.NV, 0, None, *b)
        torch.cuda.synchronize()
        val = lambda z: fp4.values(*fp4.quantize(z, fp4.NV), fp4.NV)  # noqa: E731
        return (b[0], b[1], val(v)), (b[2], b[3], val(v.T))

    (xr, xc), (wr, wc), (dr, dc) = both(x), both(w), both(dy)
    for a, b, m, n, k in ((xr, wc, M, N, K), (dr, wr, M, K, N), (xc, dc, K, N, M)):
        want, mag = fp4.scaled_mm(a[2], b[2])
        got = product(g, a, b, m, n, k, fp4.NV, True)
        assert (np.abs(got - want) <= (k / 64 + 2) * 2.0 ** -22 * mag).all()
