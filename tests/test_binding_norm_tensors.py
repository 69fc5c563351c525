"""What the binding makes of tensors given to the norms' argument blocks: their pitches, and a refusal where a type, a size or
strides would be read as something else. No GPU: nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32
T, D = 6, 64


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def norm(g, tokens=T, width=D, stream=0, block=0, **kw):
    return g.block_norm(tokens, width, stream, block, post=1, pre=1, **kw)


def test_pitches(g):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    f = norm(g, r=z(T, D), o=z(T, 80)[:, :D], r_out=z(2 * T, D)[::2], h=z(T, 100), gate=z(D), gate_rows=T)
    assert (f.ld_r, f.ld_o, f.ld_r_out, f.ld_h, f.ld_gate) == (D, 80, 2 * D, 100, D)
    assert norm(g, gate=z(1, D + 1)[:, :D], gate_rows=1 << 62).ld_gate == D
    assert norm(g, gate=z(3, D + 8)[:, :D], gate_rows=2).ld_gate == D + 8
    assert norm(g, tokens=1, r=z(D)).ld_r == D and norm(g, tokens=1, r=z(1, 2 * D).as_strided((1, D), (7, 1))).ld_r == D
    assert norm(g, width=1, r=z(T, 3)[:, :1]).ld_r == 3  # one column: no elements next to each other
    assert g.block_norm_grad(dh=z(T, 80)[:, :D], do=z(T, D)).ld_dh == 80
    # by hand, as it is
    assert norm(g, r=z(T * 70), ld_r=70).ld_r == 70 and norm(g, r=0x1000, ld_r=9).ld_r == 9


@pytest.mark.parametrize("name", ["r", "r_out", "o", "h", "gate"])
def test_matrices_that_are_something_else(g, name):
    more = {"gate_rows": 3} if name == "gate" else {}
    rows = 2 if name == "gate" else T
    bad = [torch.zeros(rows, 2 * D, dtype=BF)[:, ::2], torch.zeros(D, rows, dtype=BF).t(), torch.zeros(rows - 1, D, dtype=BF), torch.zeros(rows, D - 1, dtype=BF),
           torch.zeros(1, rows, D, dtype=BF), torch.zeros(rows * D, dtype=BF), torch.zeros((), dtype=BF)]
    for x in bad:
        with pytest.raises(ValueError) as e:
            norm(g, **{name: x}, **more)
        assert name in str(e.value)
    for dt in (torch.float16, F32, torch.int16):
        with pytest.raises(TypeError) as e:
            norm(g, **{name: torch.zeros(rows, D, dtype=dt)}, **more)
        assert name in str(e.value)
        with pytest.raises(TypeError):  # (the type also where the pitch is by hand)
            norm(g, **{name: torch.zeros(rows, D, dtype=dt), "ld_" + name: D}, **more)
    norm(g, stream=1, block=1, **{name: torch.zeros(rows, D, dtype=F32)}, **more)


def test_vectors_that_are_something_else(g):
    for name, n in (("w_post", D), ("b_post", D), ("w_pre", D), ("b_pre", D), ("res_scale", 1), ("h_scale", 1), ("stat_post", 2 * T), ("stat_pre", 2 * T)):
        norm(g, **{name: torch.zeros(n)})
        for x, kind in ((torch.zeros(n, dtype=BF), TypeError), (torch.zeros(n, dtype=torch.float64), TypeError), (torch.zeros(n - 1), ValueError),
                        (torch.zeros(n + 1, 2)[:, 0], ValueError)):
            with pytest.raises(kind) as e:
                norm(g, **{name: x})
            assert name in str(e.value)
    q, sf = torch.zeros(T, g.fp4_row_bytes(D), dtype=torch.uint8), torch.zeros(g.fp4_scale_bytes(0, T, D), dtype=torch.uint8)
    norm(g, hq=q, hsf=sf)
    for name, x, kind in (("hq", q[1:], ValueError), ("hsf", sf[1:], ValueError), ("hq", q.view(torch.int8), TypeError), ("hq", q.float(), TypeError)):
        with pytest.raises(kind):
            norm(g, **{"hq": q, "hsf": sf, name: x})


def test_gradients_that_are_something_else(g):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    f = norm(g, r=z(T, D, dt=F32), stream=1, o=z(T, D), gate=z(2, D), gate_rows=3, r_out=z(T, D, dt=F32))
    sizes = lambda **kw: g.fp8_block_norm_bwd_workspace_bytes(f, g.block_norm_grad(**kw))  # noqa: E731
    good = dict(dh=z(T, D), dr_out=z(T, D, dt=F32), dr=z(T, D, dt=F32), do=z(T, D), dgate=z(2, D, dt=F32), dres_scale=z(1, dt=F32), dw_post=z(D, dt=F32))
    for bad, kind in ((dict(dh=z(T, 2 * D)[:, ::2]), ValueError), (dict(dh=z(T, D, dt=F32)), TypeError), (dict(dr=z(T, D)), TypeError), (dict(dr_out=z(T, D)), TypeError),
                      (dict(do=z(T - 1, D)), ValueError), (dict(do=z(T, D, dt=torch.float16)), TypeError), (dict(dgate=z(1, D, dt=F32)), ValueError),
                      (dict(dgate=z(2, D)), TypeError), (dict(dw_pre=z(D - 1, dt=F32)), ValueError), (dict(db_pre=z(D, 2, dt=F32)[:, 0]), ValueError),
                      (dict(dres_scale=z(1, dt=torch.float64)), TypeError)):
        with pytest.raises(kind) as e:
            sizes(**{**good, **bad})
        assert next(iter(bad)) in str(e.value)
    if torch.cuda.is_available():
        assert sizes(**good) > 0
    else:
        with pytest.raises(g.Fp8Error):  # past the checks, the device is asked
            sizes(**good)
