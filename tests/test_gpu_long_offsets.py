"""The 4-bit operators and the norms around a block where offsets pass 2^31 elements: the results are the bits of the same
call on compact matrices (which the other tests hold against 64-bit sums)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
PITCH = 1 << 16  # elements between rows


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_mixed_precision_saturating_gb300 as g
    return g


def wide(x, pitch=PITCH):
    """x's values in rows `pitch` elements apart."""
    y = torch.empty(x.shape[0] * pitch, dtype=x.dtype, device="cuda").view(x.shape[0], pitch)[:, : x.shape[1]]
    y.copy_(x)
    return y


def room(rows, cols, dtype, pitch=PITCH):
    y = torch.empty(rows * pitch, dtype=dtype, device="cuda").view(rows, pitch)[:, :cols]
    y.fill_(7)
    return y


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF)


def operand(g, x, fmt):
    rows, cols = x.shape
    q = torch.zeros(rows, g.fp4_row_bytes(cols), dtype=torch.uint8, device="cuda")
    sf = torch.zeros(g.fp4_scale_bytes(fmt, rows, cols), dtype=torch.uint8, device="cuda")
    g.fp4_quantize(x, rows, cols, x.stride(0), fmt, g.FP8_SCALE_CURRENT, None, q, sf)
    return q, sf


@pytest.mark.parametrize("which", ["rows", "cols", "both"])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize(g, fmt, which):
    rows, cols = 33000, 72
    x = randn(rows, cols)
    xw = wide(x)
    got = []
    for m in (x, xw):
        u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
        q, sf = (u8(rows * g.fp4_row_bytes(cols)), u8(g.fp4_scale_bytes(fmt, rows, cols))) if which != "cols" else (None, None)
        qT, sfT = (u8(cols * g.fp4_row_bytes(rows)), u8(g.fp4_scale_bytes(fmt, cols, rows))) if which != "rows" else (None, None)
        st = g.TensorState(4) if fmt == 0 else None
        g.fp4_quantize(m, rows, cols, m.stride(0), fmt, g.FP8_SCALE_CURRENT, st, q, sf, qT, sfT)
        got.append([t for t in (q, sf, qT, sfT) if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dt,pitch", [(BF, PITCH), (F32, PITCH), (BF, PITCH + 1)])
def test_dequantize(g, dt, pitch):
    rows, cols = 33000, 72
    q, sf = operand(g, randn(rows, cols), 0)
    code = g.FP8_DT_BF16 if dt is BF else g.FP8_DT_F32
    a, b = torch.empty(rows, cols, dtype=dt, device="cuda"), room(rows, cols, dt, pitch)
    g.fp4_dequantize(q, sf, rows, cols, 0, None, a, code, cols)
    g.fp4_dequantize(q, sf, rows, cols, 0, None, b, code, pitch)
    assert torch.equal(a, b)


@pytest.mark.parametrize("m,n,pitch", [(33000, 64, PITCH), (33000, 61, PITCH), (48, 136, 1 << 26), (3, 136, 1 << 30)])
def test_product(g, m, n, pitch):
    a, b = operand(g, randn(m, 96), 0), operand(g, randn(n, 96, seed=1), 0)
    compact = (n + 7) // 8 * 8
    c = torch.empty(m, compact, dtype=BF, device="cuda")
    w = room(m, n, BF, pitch)
    g.fp4_scaled_mm(*a, *b, m, n, 96, 0, None, None, c, g.FP8_DT_BF16, compact)
    g.fp4_scaled_mm(*a, *b, m, n, 96, 0, None, None, w, g.FP8_DT_BF16, pitch)
    assert torch.equal(c[:, :n], w)


def test_product_of_a_long_operand(g):
    """B's codes pass 2^32 bytes: its last rows have the bits of a product with those rows alone."""
    m, n, k = 5, (1 << 21) + 256, 4096
    a = operand(g, randn(m, k), 0)
    x = randn(4096, k, seed=1)
    q = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(g.fp4_scale_bytes(0, n, k), dtype=torch.uint8, device="cuda")
    per = g.fp4_scale_bytes(0, 4096, k)
    for i in range(0, n, 4096):
        r = min(4096, n - i)
        g.fp4_quantize(x, r, k, k, 0, g.FP8_SCALE_CURRENT, None, q[i:], sf[i // 4096 * per:])
    c, d = torch.empty(m, n, dtype=BF, device="cuda"), torch.empty(m, 4096, dtype=BF, device="cuda")
    g.fp4_scaled_mm(*a, q, sf, m, n, k, 0, None, None, c, g.FP8_DT_BF16, n)
    g.fp4_scaled_mm(*a, *operand(g, x, 0), m, 4096, k, 0, None, None, d, g.FP8_DT_BF16, 4096)
    assert torch.equal(c[:, : n // 4096 * 4096].reshape(m, -1, 4096), d[:, None].expand(m, n // 4096, 4096))
    assert torch.equal(c[:, n // 4096 * 4096:], d[:, : n % 4096])


@pytest.mark.parametrize("D,stream,pitch", [(64, BF, PITCH), (512, BF, PITCH), (512, F32, PITCH), (67, BF, PITCH + 1), (8200, BF, PITCH)])
def test_norms(g, D, stream, pitch):
    T = 33000
    names = dict(r=randn(T, D).to(stream), o=randn(T, D, seed=1), dh=randn(T, D, seed=2), dr_out=randn(T, D, seed=3).to(stream))
    w, b = randn(D, seed=4).float(), randn(D, seed=5).float()
    sd = g.FP8_DT_F32 if stream is F32 else g.FP8_DT_BF16
    results = []
    for far in (False, True):
        put = (lambda x: wide(x, pitch)) if far else (lambda x: x)
        new = (lambda dt: room(T, D, dt, pitch)) if far else (lambda dt: torch.empty(T, D, dtype=dt, device="cuda"))
        ld = pitch if far else D
        x = {k: put(v) for k, v in names.items()}
        r_out, h, dr, do = new(stream), new(BF), new(stream), new(BF)
        pre = torch.empty(T, 2, device="cuda")
        post = torch.empty(T, 2, device="cuda")
        grads = {k: torch.empty(D, device="cuda") for k in ("dw_post", "db_post", "dw_pre", "db_pre")}
        f = g.block_norm(T, D, sd, g.FP8_DT_BF16, g.FP8_NORM_RMS, g.FP8_NORM_LAYER, r=x["r"], ld_r=ld, o=x["o"], ld_o=ld, w_post=w, b_post=b,
                         w_pre=w, b_pre=b, r_out=r_out, ld_r_out=ld, h=h, ld_h=ld, stat_pre=pre, stat_post=post)
        g.fp8_block_norm_fwd(f)
        d = g.block_norm_grad(dh=x["dh"], ld_dh=ld, dr_out=x["dr_out"], ld_dr_out=ld, dr=dr, ld_dr=ld, do=do, ld_do=ld, **grads)
        n = g.fp8_block_norm_bwd_workspace_bytes(f, d)
        g.fp8_block_norm_bwd(f, d, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
        results.append([r_out.clone(), h.clone(), pre, post, dr.clone(), do.clone(), *grads.values()])
        del x, r_out, h, dr, do, f, d
        torch.cuda.empty_cache()
    assert all(torch.equal(a, c) for a, c in zip(*results))
