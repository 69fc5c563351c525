"""The norms around a block on the GPU, forward and backward, against the fp64 oracle.

Bounds, with u = 2^-24: a row's statistic sums D squares in fp32 (at most D / 256 + 16 roundings in
sequence, all of one sign), so 1 / root is within (D / 512 + 16) u of itself; every output then takes
fewer than 16 roundings of terms whose magnitudes are summed alongside, and one rounding to its type.
A column sum of T terms takes at most T roundings: T u of its magnitude sum."""
import numpy as np
import pytest
import torch

from datagen import f32_from_bf16_bits
from oracle import fp4, norm

from gpu_util import host_u8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}  # unit roundoff 2^-p: significands of 8 and 24 bits


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def put(x, dt, pad=0):
    """x on the device in a matrix with `pad` more columns of 3s; and its rounded values in fp64."""
    t = torch.full((x.shape[0], x.shape[1] + pad), 3.0, dtype=DT[dt], device="cuda")
    t[:, : x.shape[1]] = torch.from_numpy(x).to(DT[dt])
    v = t[:, : x.shape[1]]
    return v, v.double().cpu().numpy()


class Case:
    def __init__(self, g, T, D, stream="bf16", block="bf16", post=1, pre=1, rows=0, alpha=True, o=True, wb=True, pad=0, seed=0, mean=0.0):
        rng = np.random.default_rng(seed + T * 3 + D)
        self.__dict__.update(g=g, T=T, D=D, stream=stream, block=block, post=post if o else 0, pre=pre, rows=rows if o else 0, pad=pad, eps=1e-5)
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.r, self.vr = put(n(T, D) * np.exp(n(1, D) * 0.3) + mean, stream, pad)
        self.o, self.vo = put(0.7 * n(T, D) + 0.2, block, pad) if o else (None, None)
        self.gate, self.vgate = put(0.5 + 0.3 * n(-(-T // rows), D), block, pad) if self.rows else (None, None)
        vec = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()  # noqa: E731
        self.par, self.vpar = {}, {}
        for k, kind in (("post", self.post), ("pre", pre)):
            if kind and wb:
                for name, x in (("w_" + k, 1 + 0.2 * n(D)), ("b_" + k, 0.1 * n(D))):
                    self.par[name] = vec(x)
                    self.vpar[name] = self.par[name].double().cpu().numpy()
        self.valpha = float(np.float32(0.9)) if alpha else 1.0
        self.alpha = vec(np.array([0.9])) if alpha else None
        self.args = dict(gate=self.vgate, gate_rows=rows or 1, post=self.post, pre=pre, alpha=self.valpha, **self.vpar)
        self.ref = norm.forward(self.vr, self.vo, eps=self.eps, **self.args)
        self.out = lambda dt: torch.full((T, D + pad), 3.0, dtype=DT[dt], device="cuda")[:, :D]  # noqa: E731

    def plan(self, **more):
        g, dt = self.g, {"bf16": self.g.FP8_DT_BF16, "f32": self.g.FP8_DT_F32}
        return g.block_norm(self.T, self.D, dt[self.stream], dt[self.block], post=self.post, pre=self.pre, eps=self.eps, r=self.r, o=self.o, gate=self.gate,
                            gate_rows=self.rows, res_scale=self.alpha, **self.par, **more)

    def forward(self, want_codes=None, stream=None, in_place=False):
        self.stat_post, self.stat_pre = torch.zeros(self.T, 2, device="cuda"), torch.zeros(self.T, 2, device="cuda")
        self.r_out = self.r if in_place else self.out(self.stream)
        self.h = self.out(self.block)
        more = {}
        if want_codes is not None:
            self.hq = torch.full((self.T, self.g.fp4_row_bytes(self.D)), 0xA5, dtype=torch.uint8, device="cuda")
            self.hsf = torch.full((self.g.fp4_scale_bytes(want_codes, self.T, self.D),), 0xA5, dtype=torch.uint8, device="cuda")
            more = dict(hq=self.hq, hsf=self.hsf, h_fmt=want_codes)
        f = self.plan(r_out=self.r_out, h=self.h, stat_post=self.stat_post, stat_pre=self.stat_pre, **more)
        torch.cuda.synchronize()
        self.g.fp8_block_norm_fwd(f, stream)
        torch.cuda.synchronize()
        return f


def rel_stat(c):
    return (c.D / 512 + 16) * U


def terms(c):
    """Magnitudes of what r' and h are summed from."""
    a = np.abs(c.vr * c.valpha)
    if c.vo is not None:
        m, i = c.ref["post"]
        n = (np.abs(c.vo) + np.abs(m)) * i * np.abs(c.vpar.get("w_post", 1.0)) + np.abs(c.vpar.get("b_post", 0.0))
        gr = norm.gate_rows_of(c.vgate, c.rows, c.T) if c.rows else 1.0
        a = a + np.abs(gr) * n
    m, i = c.ref["pre"]
    return a, (a + np.abs(m)) * i * np.abs(c.vpar.get("w_pre", 1.0)) + np.abs(c.vpar.get("b_pre", 0.0))


def check_forward(c):
    ar, ah = terms(c)
    e = rel_stat(c)
    # a mean is off by e of the mean magnitude; r' carries e of its terms into h through its statistics
    r, h = c.r_out.double().cpu().numpy(), c.h.double().cpu().numpy()
    br = 2 * e * ar + HALF[c.stream] * np.abs(c.ref["r"]) * 1.01 + 2 * e * ar.mean(axis=1, keepdims=True)
    assert (np.abs(r - c.ref["r"]) <= br).all()
    spread = (ar.mean(axis=1, keepdims=True) * c.ref["pre"][1]) if c.pre else 0.0
    bh = 6 * e * (ah + np.abs(c.ref["h"]) * (1 + spread) + spread * np.abs(c.vpar.get("w_pre", 1.0))) + HALF[c.block] * np.abs(c.ref["h"]) * 1.01
    assert (np.abs(h - c.ref["h"]) <= bh).all(), (np.abs(h - c.ref["h"]) / bh).max()
    if c.post:
        s = c.stat_post.double().cpu().numpy()
        assert np.allclose(s[:, 1:], c.ref["post"][1], rtol=4 * e, atol=0)
        assert (np.abs(s[:, :1] - c.ref["post"][0]) <= e * np.abs(c.vo).mean(axis=1, keepdims=True)).all()
    for full in (c.r_out, c.h):
        if c.pad and full is not c.r:
            base = full.as_strided((c.T, c.D + c.pad), (c.D + c.pad, 1))
            assert (base[:, c.D:] == 3.0).all()


SIZES = [(1, 1), (1, 4096), (2, 33), (3, 256), (5, 1537), (7, 768), (300, 96), (3, 8192), (2, 16384), (2, 20000), (1000, 64), (33, 2048), (64, 1032)]


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("stream,block", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_forward_sizes_and_types(g, T, D, stream, block):
    c = Case(g, T, D, stream, block, post=1, pre=2, rows=2, pad=0)
    c.forward()
    check_forward(c)


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("rows", [0, 1, 3, 1 << 40])
def test_forward_kinds_and_gates(g, post, pre, rows):
    for D, pad in ((512, 0), (200, 24), (131, 5)):
        for alpha, wb in ((True, True), (False, False)):
            c = Case(g, 10, D, "bf16", "bf16", post, pre, rows, alpha, wb=wb, pad=pad)
            c.forward()
            check_forward(c)


@pytest.mark.parametrize("D", [64, 131, 4096])
def test_forward_without_a_block(g, D):
    c = Case(g, 9, D, o=False, pre=1)
    c.forward()
    check_forward(c)


@pytest.mark.parametrize("D", [256, 333, 4096])
def test_forward_in_place_and_on_another_stream(g, D):
    c = Case(g, 50, D, "f32", "bf16", 1, 1, 7)
    s = torch.cuda.Stream()
    c.forward(stream=s, in_place=True)
    check_forward(c)


def test_large_mean_does_not_cancel(g):
    """A layer norm of rows whose mean is 300 times their spread."""
    c = Case(g, 6, 2048, "f32", "f32", 0, 2, 0, False, mean=300.0)
    c.forward()
    # the statistics' own bound, times the ratio of mean to spread that the subtraction brings in
    h = c.h.double().cpu().numpy()
    assert (np.abs(h - c.ref["h"]) <= 300 * 40 * U * (1 + np.abs(c.ref["h"]))).all()


def test_not_a_number_stays_in_its_row(g):
    for D in (512, 131):
        c = Case(g, 8, D, "bf16", "bf16", 1, 1, 0)
        c.o[2, 5] = float("nan")
        c.r[4, 7] = float("inf")
        c.forward()
        h = c.h.float().cpu().numpy()
        assert np.isnan(h[2]).all() and np.isnan(h[4, 7]) and np.isfinite(np.delete(h, [2, 4], axis=0)).all()


def test_rows_of_zeros(g):
    for D in (256, 77):
        c = Case(g, 4, D, "bf16", "bf16", 1, 2, 0, wb=False)
        c.r[1] = 0
        c.o[1] = 0
        c.forward()
        assert (c.h[1] == 0).all() and (c.r_out[1] == 0).all()


@pytest.mark.parametrize("fmt", [fp4.NV, fp4.MX])
@pytest.mark.parametrize("T,D", [(1, 32), (1, 4096), (5, 96), (130, 512), (129, 1568), (3, 16384), (2, 20000)])
@pytest.mark.parametrize("stream,block", [("bf16", "bf16"), ("f32", "f32")])
def test_forward_into_4_bits(g, fmt, T, D, stream, block):
    """The operand written for the next product: its padding exactly; its values where the oracle's h is further
    than h's own bound from every boundary between codes (elsewhere the neighbour is as good); scales likewise."""
    c = Case(g, T, D, stream, block, 1, 1, 3)
    c.forward(want_codes=fmt)
    check_forward(c)
    codes, byte = fp4.unpack(host_u8(c.hq), host_u8(c.hsf), fmt, T, D)
    fill = host_u8(c.hsf).copy()
    off = fp4.scale_offsets(fmt, T, D)
    fill[off] = fp4.FILL[fmt]
    assert (fill == fp4.FILL[fmt]).all()
    h = c.ref["h"]
    want_codes, want_byte = fp4.quantize(h.astype(np.float32), fmt)
    _, ah = terms(c)
    eps = 40 * rel_stat(c)  # relative to the row's magnitudes
    # scales: equal, or the amax lies within the bound of a rounding boundary of the scale
    for bump in (1 - eps, 1 + eps):
        _, b = fp4.quantize((h * bump).astype(np.float32), fmt)
        want_byte = np.where(byte == want_byte, want_byte, b)
    assert np.array_equal(byte, want_byte)
    # codes under the scales that were written
    scale = np.repeat(fp4.scale_value(byte, fmt), fp4.GROUP[fmt], axis=1)
    with np.errstate(all="ignore"):
        z = np.where(scale > 0, h / scale, 0.0)
        slack = np.where(scale > 0, eps * (ah + np.abs(h)) / scale, 0.0)
    low, high = fp4.code_values(fp4.cast_e2m1(z - slack)), fp4.code_values(fp4.cast_e2m1(z + slack))
    got = fp4.code_values(codes)
    assert ((got >= low) & (got <= high)).all()
    assert (codes == want_codes).mean() > 0.999


def test_4_bits_with_a_tensor_scale_and_without_h(g):
    c = Case(g, 20, 256, "bf16", "bf16", 1, 1, 0)
    s = torch.tensor([32.0], device="cuda")
    q = torch.zeros(20, g.fp4_row_bytes(256), dtype=torch.uint8, device="cuda")
    outs = []
    for scale in (None, s):
        sf = torch.zeros(g.fp4_scale_bytes(fp4.NV, 20, 256), dtype=torch.uint8, device="cuda")
        f = c.plan(r_out=c.out("bf16"), hq=q, hsf=sf, h_fmt=fp4.NV, h_scale=scale)
        g.fp8_block_norm_fwd(f)
        y = torch.zeros(20, 256, device="cuda")
        inv = torch.tensor([1.0 / 32.0], device="cuda") if scale is not None else None
        g.fp4_dequantize(q, sf, 20, 256, fp4.NV, inv, y, g.FP8_DT_F32, 256)
        outs.append(y.cpu().numpy())
    # a power of two moves every scale by five exponents and no mantissa (none is subnormal here)
    assert np.array_equal(outs[0], outs[1])


# many rows: the kernel with rows ahead in shared memory (more than two rows per SM, 1024 to 8192 columns, rows of whole 16 bytes)
@pytest.mark.parametrize("D", [1024, 1032, 1536, 2048, 3000, 4096, 4104, 5120, 6144, 6152, 8192, 8184])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_forward_many_rows(g, D, stream):
    for T, post, pre, rows, wb, pad in ((305, 1, 1, 0, True, 0), (701, 2, 2, 100, True, 8), (1001, 1, 1, 1 << 40, False, 0), (457, 0, 2, 1, True, 0), (913, 2, 0, 0, False, 8)):
        c = Case(g, T, D, stream, "bf16", post, pre, rows, wb=wb, pad=pad)
        c.forward()
        check_forward(c)


@pytest.mark.parametrize("D", [1024, 5120, 8192])
def test_forward_many_rows_f32(g, D):
    for post, pre, rows in ((1, 1, 0), (2, 2, 7)):
        c = Case(g, 500, D, "f32", "f32", post, pre, rows)
        c.forward()
        check_forward(c)


@pytest.mark.parametrize("fmt", [fp4.NV, fp4.MX])
@pytest.mark.parametrize("T,D", [(400, 1024), (333, 4096), (310, 5120), (321, 8192), (500, 1056)])
def test_many_rows_into_4_bits(g, fmt, T, D):
    test_forward_into_4_bits(g, fmt, T, D, "bf16", "bf16")


# more than 8 rows per SM (narrow rows: 32), where the rows ahead begin to pay
@pytest.mark.parametrize("T,D", [(1217, 1024), (1301, 1032), (1400, 2048), (1217, 3000), (1300, 4096), (1217, 4104), (1250, 5120), (1217, 6152), (1300, 8192), (4865, 768), (5000, 520)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_forward_rows_ahead(g, T, D, stream):
    for post, pre, rows, wb, pad in ((1, 1, 1 << 40, False, 0), (2, 2, 100, True, 8)):
        c = Case(g, T, D, stream, "bf16", post, pre, rows, wb=wb, pad=pad)
        c.forward()
        check_forward(c)


@pytest.mark.parametrize("post,pre,rows,wb", [(0, 2, 1, True), (2, 0, 0, False), (1, 2, 0, True), (0, 1, 0, False), (1, 0, 300, True)])
def test_kinds_with_rows_ahead(g, post, pre, rows, wb):
    c = Case(g, 1500, 1536, "bf16", "bf16", post, pre, rows, wb=wb, alpha=False)
    c.forward()
    check_forward(c)


@pytest.mark.parametrize("T,D", [(1217, 1024), (1250, 5120), (1300, 8192)])
def test_f32_rows_ahead(g, T, D):
    c = Case(g, T, D, "f32", "f32", 2, 1, 7)
    c.forward()
    check_forward(c)


@pytest.mark.parametrize("fmt", [fp4.NV, fp4.MX])
@pytest.mark.parametrize("T,D", [(1300, 1056), (1217, 4096), (1217, 5120), (4870, 768)])
def test_rows_ahead_into_4_bits(g, fmt, T, D):
    test_forward_into_4_bits(g, fmt, T, D, "bf16", "bf16")


def test_forward_many_rows_in_place(g):
    c = Case(g, 2000, 2048, "bf16", "bf16", 1, 1, 300)
    plan = c.plan(r_out=c.out("bf16"), h=c.out("bf16"))
    g.fp8_block_norm_fwd(plan)
    r, h = c.r.clone(), c.out("bf16")
    f = g.block_norm(c.T, c.D, g.FP8_DT_BF16, g.FP8_DT_BF16, post=1, pre=1, eps=c.eps, r=r, ld_r=c.D, o=c.o, ld_o=c.D, gate=c.gate, ld_gate=c.D, gate_rows=300,
                     res_scale=c.alpha, r_out=r, ld_r_out=c.D, h=h, ld_h=c.D, **c.par)
    g.fp8_block_norm_fwd(f)
    out = c.out("bf16"), c.out("bf16")
    g.fp8_block_norm_fwd(c.plan(r_out=out[0], h=out[1]))
    assert torch.equal(r, out[0]) and torch.equal(h, out[1])


# ------------------------------------------------------------------------------------------------
# backward
# ------------------------------------------------------------------------------------------------
def run_backward(c, dh=True, dr_out=True, want=None, stream=None, in_place=False):
    g, T, D = c.g, c.T, c.D
    rng = np.random.default_rng(T + D)
    c.forward()
    c.dh, c.vdh = put(0.1 * rng.standard_normal((T, D)), c.block, c.pad) if dh else (None, None)
    c.dro, c.vdro = put(0.1 * rng.standard_normal((T, D)) + 0.01, c.stream, c.pad) if dr_out else (None, None)
    f = c.plan(r_out=c.r_out, stat_post=c.stat_post, stat_pre=c.stat_pre)
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    outs = {"dr": c.dro if in_place else c.out(c.stream)}
    if c.o is not None:
        outs["do"] = c.out(c.block)
    if c.gate is not None:
        outs["dgate"] = new(c.gate.shape[0], D)
    if c.alpha is not None:
        outs["dres_scale"] = new(1)
    for k, kind in (("post", c.post), ("pre", c.pre)):
        if kind:
            outs["dw_" + k], outs["db_" + k] = new(D), new(D)
    if want is not None:
        outs = {k: v for k, v in outs.items() if k in want}
    b = g.block_norm_grad(dh=c.dh, dr_out=c.dro, **outs)
    n = g.fp8_block_norm_bwd_workspace_bytes(f, b)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g.fp8_block_norm_bwd(f, b, ws, n, stream)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xFF).all()
    return outs


def check_backward(c, outs):
    st = lambda t: (t.double().cpu().numpy()[:, :1], t.double().cpu().numpy()[:, 1:])  # noqa: E731
    ones = (np.zeros((c.T, 1)), np.ones((c.T, 1)))
    args = dict(gate=c.vgate, gate_rows=c.rows or 1, post=c.post, pre=c.pre, alpha=c.valpha, **c.vpar)
    vro = c.r_out.double().cpu().numpy()
    sp, sq = st(c.stat_post) if c.post else ones, st(c.stat_pre) if c.pre else ones
    ref = norm.backward(c.vr, vro, c.vdh, c.vdro, c.vo, st_post=sp, st_pre=sq, **args)
    e = rel_stat(c)
    # magnitudes: |dy w| and |z| as they enter the sums
    zp = np.abs((vro - sq[0]) * sq[1]) if c.pre else 0.0
    dz = np.abs(c.vdh * c.vpar.get("w_pre", 1.0)) if c.vdh is not None else np.zeros((c.T, c.D))
    mag = (np.abs(c.vdro) if c.vdro is not None else 0.0) + sq[1] * (dz + zp * (dz * zp).mean(axis=1, keepdims=True) + dz.mean(axis=1, keepdims=True)) if c.pre \
        else (np.abs(c.vdro) if c.vdro is not None else 0.0) + dz
    tol = {"dr": (e * 4 * mag * abs(c.valpha) + HALF[c.stream] * 1.01 * np.abs(ref["dr"]))}
    n = c.T * U + 4 * e
    tol["dw_pre"] = n * (np.abs(c.vdh) * (zp + U)).sum(axis=0) * 2 if c.vdh is not None else np.zeros(c.D)
    tol["db_pre"] = n * np.abs(c.vdh).sum(axis=0) if c.vdh is not None else np.zeros(c.D)
    tol["dres_scale"] = 8 * e * (mag * np.abs(c.vr)).sum()
    if c.vo is not None:
        gr = np.abs(norm.gate_rows_of(c.vgate, c.rows, c.T)) if c.rows else 1.0
        zo = np.abs((c.vo - sp[0]) * sp[1])
        dn = mag * gr
        dzo = dn * np.abs(c.vpar.get("w_post", 1.0))
        tol["dw_post"], tol["db_post"] = 2 * n * (dn * (zo + U)).sum(axis=0), 2 * n * dn.sum(axis=0)
        md = sp[1] * (dzo + zo * (dzo * zo).mean(axis=1, keepdims=True) + dzo.mean(axis=1, keepdims=True)) if c.post else dn
        tol["do"] = 8 * e * md + HALF[c.block] * 1.01 * np.abs(ref["do"])
        if c.rows:
            t = mag * (zo * np.abs(c.vpar.get("w_post", 1.0)) + np.abs(c.vpar.get("b_post", 0.0)))
            tol["dgate"] = np.zeros(c.vgate.shape)
            np.add.at(tol["dgate"], np.arange(c.T) // c.rows, 2 * n * t)
    ref["dres_scale"] = ref["dscale"]
    for k, v in outs.items():
        got = v.double().cpu().numpy()
        d = np.abs(got - ref[k])
        assert (d <= tol[k] + 1e-30).all(), (k, float((d / (tol[k] + 1e-30)).max()))
        if k in ("dr", "do") and c.pad and v is not c.dro:
            assert (v.as_strided((c.T, c.D + c.pad), (c.D + c.pad, 1))[:, c.D:] == 3.0).all()


@pytest.mark.parametrize("T,D", SIZES + [(3000, 128), (1500, 1024)])
@pytest.mark.parametrize("stream,block", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_backward_sizes_and_types(g, T, D, stream, block):
    c = Case(g, T, D, stream, block, post=1, pre=2, rows=5)
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("rows", [0, 1, 3, 40, 1 << 40])
def test_backward_kinds_and_gates(g, post, pre, rows):
    for T, D, pad in ((41, 256, 0), (700, 64, 8), (10, 131, 5)):
        c = Case(g, T, D, "f32", "bf16", post, pre, rows, pad=pad)
        check_backward(c, run_backward(c))


@pytest.mark.parametrize("T,D", [(913, 40), (2500, 64), (800, 520), (701, 2048), (650, 2056), (500, 4096), (333, 8192), (640, 1025), (320, 8200)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_backward_many_rows(g, T, D, stream):
    for post, pre, rows, pad in ((1, 1, 1 << 40, 0), (2, 2, 100, 8)):
        c = Case(g, T, D, stream, "bf16", post, pre, rows, pad=pad)
        check_backward(c, run_backward(c))


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 100, 305, 306, 611, 1000, 1800, 1 << 33])
def test_gate_gradients_across_shares(g, rows):
    """Groups inside, on the border of and across the parts that the tokens are split into."""
    c = Case(g, 1831, 72, "f32", "f32", 1, 1, rows)
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("D", [128, 77])
def test_backward_with_one_gradient_in(g, D):
    for dh, dro in ((True, False), (False, True)):
        c = Case(g, 50, D, "bf16", "bf16", 1, 1, 6)
        check_backward(c, run_backward(c, dh, dro))


@pytest.mark.parametrize("want", [("dr",), ("do",), ("dw_pre",), ("dgate",), ("dres_scale",), ("dw_post", "db_post")])
def test_backward_of_what_is_wanted(g, want):
    for D in (256, 99):
        c = Case(g, 60, D, "bf16", "bf16", 2, 1, 7)
        outs = run_backward(c, want=want)
        assert set(outs) == set(want)
        check_backward(c, outs)


def test_backward_without_a_block_or_parameters(g):
    for D in (512, 100):
        c = Case(g, 30, D, "bf16", "bf16", o=False, pre=1)
        check_backward(c, run_backward(c))
        c = Case(g, 30, D, "bf16", "bf16", 1, 1, 0, False, wb=False)
        check_backward(c, run_backward(c))


def test_backward_in_place_on_another_stream_and_again(g):
    for D in (1024, 130):
        c = Case(g, 200, D, "bf16", "bf16", 1, 1, 33)
        first = {k: v.clone() for k, v in run_backward(c).items()}
        again = run_backward(c, stream=torch.cuda.Stream(), in_place=True)
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_gradients_against_differences(g):
    """dr, do, dgate and dalpha against central differences of the GPU's own fp32 forward."""
    T, D = 3, 40
    c = Case(g, T, D, "f32", "f32", 1, 2, 2)
    outs = run_backward(c)
    dh, dro = c.vdh, c.vdro

    def loss():
        c.forward()
        return (c.h.double().cpu().numpy() * dh).sum() + (c.r_out.double().cpu().numpy() * dro).sum()

    step = 2.0 ** -6
    for tensor, grad, places in ((c.r, outs["dr"], [(0, 0), (2, 39)]), (c.o, outs["do"], [(1, 3), (2, 20)]),
                                 (c.gate, outs["dgate"], [(0, 5), (1, 39)]), (c.alpha, outs["dres_scale"], [(0,)])):
        grad = grad.clone()
        for at in places:
            keep = tensor[at].item()
            tensor[at] = keep + step
            up = loss()
            tensor[at] = keep - step
            down = loss()
            tensor[at] = keep
            # truncation step^2 / 6 of third derivatives of order one; rounding T D u / step of the loss
            assert abs((up - down) / (2 * step) - grad[at].item()) < 2e-3, at


def test_empty(g):
    f = g.block_norm(0, 64, 0, 0, post=0, pre=1)
    g.fp8_block_norm_fwd(f)
    dw = torch.full((64,), 5.0, device="cuda")
    b = g.block_norm_grad(dw_pre=dw)
    assert g.fp8_block_norm_bwd_workspace_bytes(f, b) == 0
    g.fp8_block_norm_bwd(f, b, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all()
