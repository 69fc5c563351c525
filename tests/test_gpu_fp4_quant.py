"""4-bit quantise and dequantise on the GPU against the oracle, bit for bit: codes, scale bytes and
their padding, both directions, ragged sizes, strides, special values, the tensor scale's state."""
import numpy as np
import pytest
import torch

from datagen import bf16_bits_from_f32, f32_from_bf16_bits
from oracle import fp4

from gpu_util import dev_bf16, host_u8

pytestmark = pytest.mark.gpu

FMTS = [fp4.NV, fp4.MX]


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def values_of(seed, rows, cols, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1)))
    return f32_from_bf16_bits(bf16_bits_from_f32(x.astype(np.float32)))


def guarded(n):
    """A buffer of n bytes between 64 bytes of 0xA5 on either side, and the whole of it."""
    whole = torch.full((n + 128,), 0xA5, dtype=torch.uint8, device="cuda")
    return whole[64:64 + n], whole


def intact(whole):
    h = host_u8(whole)
    return (h[:64] == 0xA5).all() and (h[-64:] == 0xA5).all()


def quantize(g, x, fmt, which, st=None, mode=0, ld=None, stream=None):
    """x (numpy fp32 of bf16 values, or a device tensor) -> {"q", "sf", "qT", "sfT"} as host bytes."""
    rows, cols = x.shape
    xd = x if isinstance(x, torch.Tensor) else dev_bf16(bf16_bits_from_f32(x))
    bufs, out = {}, {}
    for name, mn, k in (("", rows, cols), ("T", cols, rows)):
        if which in (("rows" if name == "" else "cols"), "both"):
            bufs["q" + name] = guarded(mn * g.fp4_row_bytes(k))
            bufs["sf" + name] = guarded(g.fp4_scale_bytes(fmt, mn, k))
    get = lambda n: bufs[n][0] if n in bufs else None  # noqa: E731
    g.fp4_quantize(xd, rows, cols, cols if ld is None else ld, fmt, mode, st, get("q"), get("sf"), get("qT"), get("sfT"), stream)
    torch.cuda.synchronize()
    for n, (b, whole) in bufs.items():
        assert intact(whole), n
        out[n] = host_u8(b)
    return out


def check(out, x, fmt, s=np.float32(1)):
    for name, v in (("", x), ("T", x.T)):
        if "q" + name in out:
            q, sf = fp4.pack(*fp4.quantize(v, fmt, s), fmt)
            assert np.array_equal(out["sf" + name], sf), name
            assert np.array_equal(out["q" + name].reshape(q.shape), q), name


SIZES = [(1, 1), (1, 32), (1, 4096), (3, 31), (17, 16), (33, 100), (127, 129), (128, 256), (130, 1024), (257, 520), (1024, 48), (40, 2056)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_codes_and_scales(g, fmt, rows, cols):
    x = values_of(rows * 7 + cols, rows, cols)
    check(quantize(g, x, fmt, "both"), x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("which", ["rows", "cols"])
def test_one_direction(g, fmt, which):
    x = values_of(5, 200, 320)
    out = quantize(g, x, fmt, which)
    assert len(out) == 2
    check(out, x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ld,offset", [(264, 0), (257, 0), (272, 1), (264, 8)])
def test_strides_and_alignment(g, fmt, ld, offset):
    """Rows of a wider matrix, from places that are and are not 16-byte aligned."""
    big = values_of(11, 150, ld)
    dev = dev_bf16(bf16_bits_from_f32(big)).view(-1)
    rows, cols = 149, 240
    view = dev[offset:].as_strided((rows, cols), (ld, 1))
    x = big.reshape(-1)[offset:offset + rows * ld].reshape(rows, ld)[:, :cols]
    check(quantize(g, view, fmt, "both", ld=ld), x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_special_values(g, fmt):
    x = values_of(2, 96, 192, 0.5)
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 70] = -np.inf
    x[2, 71] = np.nan
    x[5] = 0.0
    x[6] = -0.0
    x[7, :64] = 1e-38
    x[8, :64] = 2.0 ** -133  # subnormal in bf16
    x[9] = 3.38e38
    x[10, ::2] = -x[10, ::2] * 1e30
    x = f32_from_bf16_bits(bf16_bits_from_f32(x))
    check(quantize(g, x, fmt, "both"), x, fmt)


def test_every_bf16_value(g):
    """All finite bf16 bit patterns as a group's largest element, among smaller ones."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    x = np.zeros((len(bits), 32), dtype=np.float32)
    x[:, 5] = f32_from_bf16_bits(bits)
    with np.errstate(all="ignore"):
        x[:, 9] = f32_from_bf16_bits(bf16_bits_from_f32((-x[:, 5] * 0.4).astype(np.float32)))
    for fmt in FMTS:
        check(quantize(g, x, fmt, "rows"), x, fmt)


@pytest.mark.parametrize("which", ["rows", "cols", "both"])
def test_tensor_scale_from_its_own_amax(g, which):
    x = values_of(21, 300, 224)
    st = g.TensorState(16)
    out = quantize(g, x, fp4.NV, which, st)
    snap, a = st.snapshot(), np.abs(x).max()
    s = np.float32(2688) / np.float32(a)
    assert snap["amax_cur"] == a and snap["scale"] == s and snap["scale_inv"] == np.float32(a) / np.float32(2688)
    assert snap["overflow"] == 0 and snap["underflow"] == 0
    check(out, x, fp4.NV, s)


def test_tensor_scale_from_a_history(g):
    st = g.TensorState(4)
    amaxes = []
    for step in range(6):
        x = values_of(step, 65, 130) * np.float32(2.0 ** (step % 3))
        out = quantize(g, x, fp4.NV, "both", st, g.FP8_SCALE_DELAYED)
        a = np.abs(x).max()
        eff = max(amaxes[-4:]) if amaxes else a  # bootstrap: its own
        s = np.float32(2688) / np.float32(eff)
        snap = st.snapshot()
        assert snap["amax_cur"] == a and snap["scale"] == s
        check(out, x, fp4.NV, s)
        g.fp8_history_commit(st)
        amaxes.append(a)


def test_zero_and_infinite_tensors_scale_by_one(g):
    for fill in (0.0, np.inf):
        x = np.full((32, 64), fill, dtype=np.float32)
        st = g.TensorState(16)
        out = quantize(g, x, fp4.NV, "both", st)
        assert st.snapshot()["scale"] == 1.0 and st.snapshot()["scale_inv"] == 1.0
        check(out, x, fp4.NV)


def test_another_stream(g):
    x = values_of(9, 512, 512)
    s = torch.cuda.Stream()
    xd = dev_bf16(bf16_bits_from_f32(x))
    torch.cuda.synchronize()
    check(quantize(g, xd, fp4.NV, "both", stream=s), x, fp4.NV)
    with torch.cuda.stream(s):
        check(quantize(g, xd, fp4.MX, "both"), x, fp4.MX)


def test_empty(g):
    for shape in ((0, 64), (64, 0)):
        g.fp4_quantize(None, *shape, 64, fp4.NV, 0, None, None, None)
        g.fp4_dequantize(None, None, *shape, fp4.NV, None, None, g.FP8_DT_F32, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mn,k", [(1, 1), (5, 31), (130, 320), (129, 1001), (64, 4096)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_dequantize(g, fmt, mn, k, dt, pad):
    """All 16 codes under finite and NaN scales; the values times the tensor's scale in fp32, rounded once."""
    rng = np.random.default_rng(mn + k + fmt)
    codes = rng.integers(0, 16, (mn, k)).astype(np.uint8)
    byte = rng.integers(90, 160, (mn, -(-k // fp4.GROUP[fmt]))).astype(np.uint8) if fmt == fp4.MX else \
        rng.integers(0, 127, (mn, -(-k // 16))).astype(np.uint8)
    byte[0, -1] = fp4.NAN_SCALE[fmt]
    q, sf = fp4.pack(codes, byte, fmt)
    d = np.float32(0.37)
    ld = k + pad
    y = torch.full((mn, ld), 7.0, dtype=torch.bfloat16 if dt == "bf16" else torch.float32, device="cuda")
    dd = torch.tensor([d], device="cuda")
    qd, sd = torch.from_numpy(q).cuda(), torch.from_numpy(sf).cuda()
    for scale_inv in (None, dd):
        g.fp4_dequantize(qd, sd, mn, k, fmt, scale_inv, y, g.FP8_DT_BF16 if dt == "bf16" else g.FP8_DT_F32, ld)
        v = fp4.values(codes, byte, fmt).astype(np.float32)
        want = torch.from_numpy(v if scale_inv is None else v * d).to(y.dtype).float().numpy()
        got = y.float().cpu().numpy()
        assert np.array_equal(np.isnan(got[:, :k]), np.isnan(want)) and np.array_equal(np.nan_to_num(got[:, :k]), np.nan_to_num(want))
        assert (got[:, k:] == 7.0).all()


def test_history_amax_ignores_nan(g):
    x = values_of(31, 140, 150)
    x[3, 4] = np.nan
    x[100, 149] = np.nan
    x = f32_from_bf16_bits(bf16_bits_from_f32(x))
    st = g.TensorState(4)
    for _ in range(2):  # from an empty history, and from one
        out = quantize(g, x, fp4.NV, "both", st, g.FP8_SCALE_DELAYED)
        assert st.snapshot()["amax_cur"] == np.nanmax(np.abs(x))
        check(out, x, fp4.NV, np.float32(2688) / np.float32(np.nanmax(np.abs(x))))
        g.fp8_history_commit(st)
