"""Heads' norm and rotation, forward and backward, against the oracle in 64 bits: both layouts, parts of the head, odd sizes, strides and
addresses, far positions, in place, no tokens.

Bounds. A rotated element is made of two products of normed values: norm (a sum of D squares, a root and three products: relative error
below (D / 32 + 12) 2^-24 under any order of the lanes' sums), a sine and a cosine with errors of 2^-22, one rounding each for the
products and their sum. Together below e = (D / 32 + 24) 2^-24 of |a| + |b|, the pair's normed magnitudes times the amplitude; the stored
value adds half a step of its type. Backward, the same for dz, and for its projection on z, whose sum of D terms is bounded by its
magnitudes; dw adds the error of a sum of n terms in the order of lanes, warps and CTAs, each partial sum below n 2^-24 of the terms'
magnitudes, with n the terms that one lane adds, and a few more levels."""
import numpy as np
import pytest
import torch

from oracle import heads

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def fractions(g, rot, base=10000.0):
    t = g.rope_turns(rot, base)
    return t, [int(x) & ((1 << 64) - 1) for x in t.cpu().tolist()]


def pairs_magnitude(x, rot, inter):
    """|a| + |b| at both members of each pair, |x| where nothing turns."""
    m = np.abs(x)
    a, b = heads._members(rot, inter)
    both = m[..., a] + m[..., b]
    m[..., a], m[..., b] = both, both
    return m


CASES = [  # T, Hq, Hk, D, rot, interleaved, norm, type, offset of the rows
    (1, 1, 1, 64, 64, False, True, torch.bfloat16, 0), (3, 32, 8, 128, 128, False, True, torch.bfloat16, 0), (37, 5, 3, 128, 64, True, True, torch.bfloat16, 0),
    (37, 12, 12, 64, 32, False, False, torch.float32, 0), (5, 7, 0, 80, 40, False, True, torch.float32, 0), (5, 0, 2, 96, 96, True, True, torch.bfloat16, 0),
    (9, 3, 1, 256, 128, False, True, torch.bfloat16, 0), (9, 3, 1, 256, 256, True, True, torch.float32, 0), (4, 2, 2, 8, 8, False, True, torch.bfloat16, 0),
    (11, 3, 2, 33, 10, False, True, torch.bfloat16, 0), (11, 3, 2, 33, 10, True, False, torch.float32, 0), (6, 2, 2, 1, 0, False, True, torch.float32, 0),
    (7, 4, 2, 128, 128, False, True, torch.bfloat16, 1), (7, 4, 2, 64, 20, False, True, torch.bfloat16, 0), (7, 4, 2, 72, 24, True, True, torch.bfloat16, 4),
    (300, 9, 3, 128, 0, False, True, torch.bfloat16, 0), (1031, 33, 9, 64, 64, True, True, torch.bfloat16, 0), (2, 2, 2, 250, 250, True, True, torch.bfloat16, 0),
]


def make(g, T, Hq, Hk, D, rot, inter, norm, dt, off, seed=0, apart=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    H = Hq + 2 * Hk
    x = torch.zeros(T * H * D + off, dtype=dt, device="cuda")
    x[off:] = (rand(T * H * D) * torch.exp(rand(T * H * D))).to(dt)
    x = x[off:].view(H, T, D).transpose(0, 1) if apart else x[off:].view(T, H, D)
    pos = (torch.arange(T, device="cuda") * 7919 % 1048576 + (2 ** 31 - 1048576 if seed == 5 else 0)).to(torch.int32)
    turns, frac = fractions(g, rot)
    w = [1 + 0.3 * rand(D) if norm else None for _ in range(2)]
    return x, pos, turns, frac, w


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("apart", [False, True])
def test_forward(g, case, apart):
    T, Hq, Hk, D, rot, inter, norm, dt, off = case
    x, pos, turns, frac, w = make(g, *case, seed=5 if apart else 1, apart=apart)
    out = torch.full((T, Hq + Hk + 1, D), 7.0, dtype=dt, device="cuda")
    f = g.qk_rope(T, Hq, Hk, D, rot, g.FP8_DT_F32 if dt == torch.float32 else g.FP8_DT_BF16, layout=int(inter), norm=int(norm), eps=1e-5, amplitude=1.2, turns=turns, pos=pos,
                  q=x[:, :Hq], k=x[:, Hq:Hq + Hk], w_q=w[0], w_k=w[1], q_out=out[:, :Hq], k_out=out[:, Hq:Hq + Hk])
    g.fp8_qk_rope_fwd(f)
    torch.cuda.synchronize()
    theta = heads.angle(pos.cpu().tolist(), frac)
    e = (D / 32 + 24) * 2.0 ** -24
    for a, b, ww in ((0, Hq, w[0]), (Hq, Hq + Hk, w[1])):
        if a == b:
            continue
        xx = f64(x[:, a:b])
        n = heads.norm(xx, None if ww is None else f64(ww), 1e-5) if norm else xx
        ref = heads.rotate(n, theta, inter, 1.2)
        bound = e * 1.2 * pairs_magnitude(n, rot, inter) + HALF[dt] * np.abs(ref) + 1e-38
        assert np.all(np.abs(f64(out[:, a:b]) - ref) <= bound)
    assert torch.all(out[:, Hq + Hk:] == 7.0)


def test_in_place_and_defaults(g):
    """Without pos token t is at position t; in place over a projection's rows, values left alone; only queries, only keys."""
    T, Hq, Hk, D = 13, 4, 2, 128
    x, _, turns, frac, w = make(g, T, Hq, Hk, D, 128, False, True, torch.bfloat16, 0)
    keep = x.clone()
    out = torch.empty(T, Hq + Hk, D, dtype=torch.bfloat16, device="cuda")
    more = dict(norm=1, turns=turns, w_q=w[0], w_k=w[1])
    g.fp8_qk_rope_fwd(g.qk_rope(T, Hq, Hk, D, 128, 0, q=x[:, :Hq], k=x[:, Hq:Hq + Hk], q_out=out[:, :Hq], k_out=out[:, Hq:], **more))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    only = torch.zeros_like(out)
    g.fp8_qk_rope_fwd(g.qk_rope(T, Hq, Hk, D, 128, 0, q=x[:, :Hq], q_out=only[:, :Hq], pos=pos, **more))
    assert torch.equal(only[:, :Hq], out[:, :Hq]) and not only[:, Hq:].any()
    g.fp8_qk_rope_fwd(g.qk_rope(T, Hq, Hk, D, 128, 0, k=x[:, Hq:Hq + Hk], k_out=only[:, Hq:], pos=pos, **more))
    assert torch.equal(only, out)
    g.fp8_qk_rope_fwd(g.qk_rope(T, Hq, Hk, D, 128, 0, q=x[:, :Hq], k=x[:, Hq:Hq + Hk], q_out=x[:, :Hq], k_out=x[:, Hq:Hq + Hk], **more))
    assert torch.equal(x[:, :Hq + Hk], out) and torch.equal(x[:, Hq + Hk:], keep[:, Hq + Hk:])


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("apart", [False, True])
def test_backward(g, case, apart):
    T, Hq, Hk, D, rot, inter, norm, dt, off = case
    x, pos, turns, frac, w = make(g, *case, seed=5 if apart else 2, apart=apart)
    dy = make(g, *case, seed=3, apart=apart)[0]
    dx = torch.full((T, Hq + Hk + 1, D), 7.0, dtype=dt, device="cuda")
    dw = [torch.full((D,), 7.0, device="cuda") if norm else None for _ in range(2)]
    f = g.qk_rope(T, Hq, Hk, D, rot, g.FP8_DT_F32 if dt == torch.float32 else g.FP8_DT_BF16, layout=int(inter), norm=int(norm), eps=1e-5, amplitude=0.8, turns=turns, pos=pos,
                  q=x[:, :Hq], k=x[:, Hq:Hq + Hk], w_q=w[0], w_k=w[1])
    b = g.qk_rope_grad(dq_out=dy[:, :Hq], dk_out=dy[:, Hq:Hq + Hk], dq=dx[:, :Hq], dk=dx[:, Hq:Hq + Hk], dw_q=dw[0], dw_k=dw[1])
    n = g.fp8_qk_rope_bwd_workspace_bytes(f, b)
    assert (n > 0) == bool(norm)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    g.fp8_qk_rope_bwd(f, b, ws, n)
    first = [t.clone() for t in [dx] + [t for t in dw if t is not None]]
    g.fp8_qk_rope_bwd(f, b, ws, n)
    assert all(torch.equal(a, c) for a, c in zip(first, [dx] + [t for t in dw if t is not None]))
    theta = heads.angle(pos.cpu().tolist(), frac)
    e = (D / 32 + 24) * 2.0 ** -24
    for a, c, ww, dww in ((0, Hq, w[0], dw[0]), (Hq, Hq + Hk, w[1], dw[1])):
        if a == c:
            assert dww is None or not dww.any()
            continue
        xx, dd = f64(x[:, a:c]), f64(dy[:, a:c])
        ref, ref_w = heads.backward(dd, xx, None if ww is None else f64(ww), 1e-5, theta, inter, 0.8, norm)
        d = 0.8 * pairs_magnitude(dd, rot, inter)  # |dn| and its error's measure
        if norm:
            r = 1 / np.sqrt((xx * xx).mean(axis=-1, keepdims=True) + 1e-5)
            z, dz = np.abs(xx * r), d * np.abs(f64(ww))
            bound = 2 * e * r * (dz + z * (dz * z).mean(axis=-1, keepdims=True)) + HALF[dt] * np.abs(ref) + 1e-38
            terms = T * (Hq + Hk)  # of one sum, at most
            assert np.all(np.abs(f64(dww) - ref_w) <= (2 * e + (terms + 64) * 2.0 ** -24) * (d * z).sum(axis=(0, 1)))
        else:
            bound = e * d + HALF[dt] * np.abs(ref) + 1e-38
        assert np.all(np.abs(f64(dx[:, a:c]) - ref) <= bound)
    assert torch.all(dx[:, Hq + Hk:] == 7.0)


def test_backward_parts(g):
    """In place, without dw, without dx, one part alone: the same numbers."""
    T, Hq, Hk, D = 21, 4, 2, 64
    x, pos, turns, _, w = make(g, T, Hq, Hk, D, 64, False, True, torch.bfloat16, 0)
    dy = make(g, T, Hq, Hk, D, 64, False, True, torch.bfloat16, 0, seed=3)[0].contiguous()
    f = g.qk_rope(T, Hq, Hk, D, 64, 0, norm=1, turns=turns, pos=pos, q=x[:, :Hq], k=x[:, Hq:Hq + Hk], w_q=w[0], w_k=w[1])

    def back(**kw):
        b = g.qk_rope_grad(**kw)
        n = g.fp8_qk_rope_bwd_workspace_bytes(f, b)
        g.fp8_qk_rope_bwd(f, b, torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n)

    dx, dwq, dwk = torch.zeros_like(x), torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    ins = dict(dq_out=dy[:, :Hq], dk_out=dy[:, Hq:Hq + Hk])
    back(dq=dx[:, :Hq], dk=dx[:, Hq:Hq + Hk], dw_q=dwq, dw_k=dwk, **ins)
    other = torch.zeros_like(x)
    back(dq=other[:, :Hq], dq_out=ins["dq_out"])
    back(dk=other[:, Hq:Hq + Hk], dk_out=ins["dk_out"])
    assert torch.equal(other, dx)
    only = torch.zeros(D, device="cuda")
    back(dw_k=only, dk_out=ins["dk_out"])
    assert torch.allclose(only, dwk, rtol=1e-4, atol=1e-4)  # (another split of the tokens)
    back(dq=dy[:, :Hq], dk=dy[:, Hq:Hq + Hk], **ins)
    assert torch.equal(dy[:, :Hq + Hk], dx[:, :Hq + Hk])


def test_nothing_to_sum(g):
    D = 64
    dwq, dwk = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    t = g.rope_turns(D, 1e4)
    f = g.qk_rope(0, 4, 2, D, D, 0, norm=1, turns=t)
    g.fp8_qk_rope_bwd(f, g.qk_rope_grad(dw_q=dwq, dw_k=dwk), None, 0)
    assert not dwq.any() and not dwk.any()


def test_a_gradient_against_differences(g):
    """The backward's dx in fp32 against differences of the forward."""
    T, D = 2, 16
    x, pos, turns, _, w = make(g, T, 1, 1, D, 8, True, True, torch.float32, 0)
    x = x / x.abs().max()
    gen = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(T, 1, D, generator=gen, device="cuda")
    dx = torch.empty_like(dy)
    more = dict(layout=1, norm=1, eps=1e-2, turns=turns, pos=pos, w_q=w[0])
    g.fp8_qk_rope_bwd(g.qk_rope(T, 1, 0, D, 8, 1, q=x[:, :1], **more), g.qk_rope_grad(dq_out=dy, dq=dx), None, 0)

    def loss(q):
        y = torch.empty_like(dy)
        g.fp8_qk_rope_fwd(g.qk_rope(T, 1, 0, D, 8, 1, q=q, q_out=y, **more))
        return float((y.double() * dy.double()).sum())

    h = 2.0 ** -8  # forward errors of 2^-21 x 16 terms over 2 h: 2^-10; the third derivative's h^2 / 6: 2^-10 with values of a few
    for i in range(T):
        for d in range(D):
            step = torch.zeros_like(x[:, :1])
            step[i, 0, d] = h
            diff = (loss(x[:, :1] + step) - loss(x[:, :1] - step)) / (2 * h)
            assert abs(diff - float(dx[i, 0, d])) < 2.0 ** -6 * (1 + float(dx.abs().max()))
