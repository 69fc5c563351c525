"""Elements that do not turn, when they are infinite or NaN: rotation, its gradient and the append leave them where they are, and every other
element keeps the bits that it has without them. Vector kernels and those of single elements (rows at odd addresses), both layouts.

With a norm an infinity makes the row's factor 0: it becomes a NaN itself and the row's other elements 0, a NaN makes the whole row NaN, and in
the gradient an infinite term of the projection on the row reaches all of its elements; there the oracle says where what stands."""
import numpy as np
import pytest
import torch

from oracle import heads
from test_gpu_qk_rope import f64, fractions

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def rows(T, H, D, dt, off, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(T * H * D + off, dtype=dt, device="cuda")
    x[off:] = torch.randn(T * H * D, generator=gen, device="cuda").to(dt)
    return x[off:].view(T, H, D)


def spoiled(x, rot, value):
    """Token t with `value` in element rot + t of every head."""
    y = torch.empty(x.numel() + x.storage_offset(), dtype=x.dtype, device="cuda")[x.storage_offset():].view(x.shape)
    y.copy_(x)
    at = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
    for t in range(x.shape[0]):
        y[t, :, rot + t] = value
        at[t, :, rot + t] = True
    return y, at


CASES = [  # D, rot, interleaved, type, offset
    (128, 64, False, torch.bfloat16, 0), (128, 64, True, torch.bfloat16, 0), (64, 24, False, torch.bfloat16, 0), (64, 22, True, torch.bfloat16, 0), (256, 128, False, torch.bfloat16, 0),
    (64, 32, False, torch.float32, 0), (128, 26, True, torch.float32, 0), (128, 0, False, torch.bfloat16, 0), (64, 0, True, torch.float32, 0),
    (128, 64, False, torch.bfloat16, 1), (64, 22, True, torch.bfloat16, 3), (33, 10, False, torch.float32, 0), (64, 20, False, torch.bfloat16, 0), (40, 0, True, torch.bfloat16, 1),
]
case_ids = [f"{d}-{r}-{'pairs' if i else 'halves'}-{str(t)[6:]}-{o}" for d, r, i, t, o in CASES]


def block(g, case, x, norm, **out):
    D, rot, inter, dt, _ = case
    turns, frac = fractions(g, rot)
    T, H = x.shape[:2]
    f = g.qk_rope(T, H - 1, 1, D, rot, int(dt == torch.float32), layout=int(inter), norm=int(norm), eps=1e-5, amplitude=1.1, turns=turns, q=x[:, : H - 1], k=x[:, H - 1:], **out)
    return f, heads.angle(range(T), frac)


@pytest.mark.parametrize("case", CASES, ids=case_ids)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_forward(g, case, value):
    D, rot, inter, dt, off = case
    x = rows(D - rot, 4, D, dt, off, 1)
    bad, at = spoiled(x, rot, value)
    outs = {}
    for name, src in (("clean", x), ("bad", bad)):
        y = torch.full_like(x, 7.0)
        f, _ = block(g, case, src, False, q_out=y[:, :3], k_out=y[:, 3:])
        g.fp8_qk_rope_fwd(f)
        outs[name] = y
        assert torch.equal(y[..., rot:].nan_to_num(nan=3.0), src[..., rot:].nan_to_num(nan=3.0))
    assert torch.equal(bits(outs["bad"])[~at], bits(outs["clean"])[~at])
    assert torch.equal(outs["bad"][at].nan_to_num(nan=3.0), bad[at].nan_to_num(nan=3.0))
    # with a norm
    y = torch.full_like(x, 7.0)
    f, _ = block(g, case, bad, True, q_out=y[:, :3], k_out=y[:, 3:])
    g.fp8_qk_rope_fwd(f)
    assert torch.all(torch.isnan(y)) if np.isnan(value) else torch.all(torch.isnan(y) == at) and torch.all(y[~at] == 0)


@pytest.mark.parametrize("case", CASES, ids=case_ids)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_gradient(g, case, value):
    D, rot, inter, dt, off = case
    x, dy = rows(D - rot, 4, D, dt, off, 1), rows(D - rot, 4, D, dt, off, 2)
    bad, at = spoiled(dy, rot, value)
    outs = {}
    for norm in (False, True):
        for name, src in (("clean", dy), ("bad", bad)):
            dx = torch.full_like(x, 7.0)
            dw = [torch.full((D,), 7.0, device="cuda") if norm else None for _ in range(2)]
            f, theta = block(g, case, x, norm)
            b = g.qk_rope_grad(dq_out=src[:, :3], dk_out=src[:, 3:], dq=dx[:, :3], dk=dx[:, 3:], dw_q=dw[0], dw_k=dw[1])
            n = g.fp8_qk_rope_bwd_workspace_bytes(f, b)
            g.fp8_qk_rope_bwd(f, b, torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n)
            outs[name] = dx, dw
        if not norm:
            assert torch.equal(bits(outs["bad"][0])[~at], bits(outs["clean"][0])[~at])
            assert torch.equal(outs["bad"][0][at].nan_to_num(nan=3.0), bad[at].nan_to_num(nan=3.0))
            continue
        with np.errstate(invalid="ignore"):
            want, _ = heads.backward(f64(bad), f64(x), None, 1e-5, theta, inter, 1.1, True)
        got = f64(outs["bad"][0])
        assert np.array_equal(np.isnan(got), np.isnan(want))
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf])
        for (a, b_), z in zip(zip(outs["bad"][1], outs["clean"][1]), (x[:, :3], x[:, 3:])):
            # every element that does not turn has had the value once per head; the others' sums are the same ones
            assert torch.equal(bits(a[:rot]), bits(b_[:rot]))
            if np.isnan(value):
                assert torch.all(torch.isnan(a[rot:]))
            else:
                signs = torch.stack([torch.sign(z[t, :, rot + t].float()) for t in range(D - rot)])
                same = signs.abs().sum(1) == signs.sum(1).abs()
                assert torch.equal(a[rot:][same], (value * signs.sum(1))[same]) and torch.all(torch.isnan(a[rot:][~same]))


@pytest.mark.parametrize("case", CASES, ids=case_ids)
def test_a_copy_without_a_norm(g, case):
    """What does not turn comes through by the bit, zeros of both signs and the smallest numbers among it, forward and backward."""
    D, rot, inter, dt, off = case
    x = rows(9, 4, D, dt, off, 1)
    x[::2, :, rot:] *= torch.randint(0, 2, (5, 4, D - rot), device="cuda").to(dt)  # (a product: -0 where x is negative)
    x[1, :, rot:] *= 2.0 ** -126
    assert torch.any(bits(x[..., rot:]) == bits(torch.tensor([-0.0], dtype=dt, device="cuda")))
    y, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    f, _ = block(g, case, x, False, q_out=y[:, :3], k_out=y[:, 3:])
    g.fp8_qk_rope_fwd(f)
    g.fp8_qk_rope_bwd(f, g.qk_rope_grad(dq_out=x[:, :3], dk_out=x[:, 3:], dq=dx[:, :3], dk=dx[:, 3:]), None, 0)
    for out in (y, dx):
        assert torch.equal(bits(out[..., rot:].contiguous()), bits(x[..., rot:].contiguous()))


@pytest.mark.parametrize("D, rot, inter, off", [(128, 64, False, 0), (128, 64, True, 0), (64, 32, False, 1), (96, 32, True, 3), (128, 0, False, 0), (64, 0, True, 1), (256, 128, False, 0)])
@pytest.mark.parametrize("mx", [False, True])
def test_append(g, D, rot, inter, off, mx):
    """A token of each value, in the last group of 32 of its heads. In 8 bits an infinity saturates, and its group's power of two is the largest;
    a NaN makes its group NaN; the other groups keep their bytes."""
    Hq, Hk, page, values = 3, 2, 8, (INF, -INF, NAN)
    T = len(values)
    turns, _ = fractions(g, rot)
    got = []
    for spoil in (False, True):
        x = rows(T, Hq + 2 * Hk, D, torch.bfloat16, off, 4)
        if spoil:
            for t, value in enumerate(values):
                x[t, :, D - 3] = value
        cache = [torch.zeros(1, Hk, page, D, dtype=torch.uint8 if mx else torch.bfloat16, device="cuda") for _ in range(2)]
        units = [torch.zeros(1, Hk, page, D // 32, dtype=torch.uint8, device="cuda") for _ in range(2)] if mx else []
        q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        f = g.qk_rope(T, Hq, Hk, D, rot, 0, layout=int(inter), amplitude=1.1, turns=turns, q=x[:, :Hq], k=x[:, Hq:Hq + Hk], v=x[:, Hq + Hk:], q_out=q_out)
        batch = g.kv_batch(T, *(torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [T], [[0]])))
        g.fp8_kv_append(f, g.kv_cache(*cache, *units), batch)
        got.append((q_out, cache, units))
    torch.cuda.synchronize()
    (q0, cache0, units0), (q1, cache1, units1) = got
    others = torch.arange(D, device="cuda") != D - 3
    assert torch.equal(bits(q0[..., others]), bits(q1[..., others]))
    for t, value in enumerate(values):
        assert torch.all(q1[t, :, D - 3] == value) if value == value else torch.all(torch.isnan(q1[t, :, D - 3]))
    for i in range(2):
        a, b = cache0[i][0, :, :T], cache1[i][0, :, :T]
        if not mx:
            assert torch.equal(bits(a[..., others]), bits(b[..., others]))
            for t, value in enumerate(values):
                assert torch.all(b[:, t, D - 3] == value) if value == value else torch.all(torch.isnan(b[:, t, D - 3]))
            continue
        assert torch.equal(a[..., : D - 32], b[..., : D - 32]) and torch.equal(units0[i][0, :, :T, :-1], units1[i][0, :, :T, :-1])
        last, last_units = b[..., D - 32:], units1[i][0, :, :T, -1]
        assert torch.all(last_units == torch.tensor([247, 247, 255], dtype=torch.uint8, device="cuda"))
        # 448 * 2^120 and its negative; the others of the group are below half of the smallest step there
        assert torch.all(last[:, 0, 29] == 0x7E) and torch.all(last[:, 1, 29] == 0xFE)
        assert not (last[:, 2] & 127).any() and not (last[:, :2, others[D - 32:]] & 127).any()


@pytest.mark.parametrize("case", CASES, ids=case_ids)
@pytest.mark.parametrize("norm", [False, True])
def test_in_place_and_captured(g, case, norm):
    """Heads that turn in part over their own rows, forward and gradient, from a graph: the bits of calls with an output of their own."""
    D, rot, inter, dt, off = case
    x, dy = rows(70, 5, D, dt, off, 1), rows(70, 5, D, dt, off, 2)
    work, back = (torch.empty(x.numel() + off, dtype=dt, device="cuda")[off:].view(x.shape) for _ in range(2))
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(2, 2, D, device="cuda")
    kw = lambda i: dict(dw_q=dw[i, 0], dw_k=dw[i, 1]) if norm else {}  # noqa: E731
    f, _ = block(g, case, x, norm, q_out=y[:, :4], k_out=y[:, 4:])
    f_in, _ = block(g, case, work, norm, q_out=work[:, :4], k_out=work[:, 4:])
    b = g.qk_rope_grad(dq_out=dy[:, :4], dk_out=dy[:, 4:], dq=dx[:, :4], dk=dx[:, 4:], **kw(0))
    b_in = g.qk_rope_grad(dq_out=back[:, :4], dk_out=back[:, 4:], dq=back[:, :4], dk=back[:, 4:], **kw(1))
    n = g.fp8_qk_rope_bwd_workspace_bytes(f, b)
    ws = [torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    g.fp8_qk_rope_fwd(f)
    g.fp8_qk_rope_bwd(f, b, ws[0], n)
    g.fp8_qk_rope_fwd(f_in)  # (the first call of the capture's kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.fp8_qk_rope_fwd(f_in)
        g.fp8_qk_rope_bwd(f, b_in, ws[1], n)
    for _ in range(2):
        work.copy_(x)
        back.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(work), bits(y)) and torch.equal(bits(back), bits(dx))
        assert not norm or torch.equal(dw[0], dw[1])
