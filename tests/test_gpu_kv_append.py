"""Appending keys and values to a paged cache against the oracle: both formats and layouts, ragged batches, pages in any order, rows of
nobody, places out of range, unusual values. What is not written keeps its bytes.

Bounds: bf16 as in the heads' forward (tests of the rotation: (D / 32 + 24) 2^-24 of the pair's magnitudes before rounding, then half a
step, 2^-8 of the value). In 8 bits an element is off by half a step of E4M3, 2^-4 of its value or 2^-10 of the group's unit, plus
that error; where the group's largest magnitude is within the error of a boundary, the unit may be the next one, whose steps are twice as large."""
import numpy as np
import pytest
import torch

from oracle import heads
from test_gpu_qk_rope import f64, fractions, pairs_magnitude

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """Sequences of `new` tokens that end at `total`; T rows, some of them nobody's; a cache full of a sentinel."""

    def __init__(self, g, new, total, Hq, Hk, D, page, mx, inside, extra=2, seed=0, off=0):
        self.new, self.total, self.page, self.mx = new, total, page, mx
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.T = sum(new) + extra
        need = [-(-t // page) for t in total]
        self.pages, width = sum(need) + 2, max(need) + 1
        order = torch.randperm(self.pages, generator=gen, device="cuda").cpu().tolist()
        self.table = np.full((len(new), width), -7, dtype=np.int32)
        for s, n in enumerate(need):
            self.table[s, :n] = [order.pop() for _ in range(n)]
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.array(total, dtype=np.int32)
        x = torch.zeros(self.T * (Hq + 2 * Hk) * D + off, dtype=torch.bfloat16, device="cuda")
        x[off:] = (rand(x.numel() - off) * torch.exp(rand(x.numel() - off))).to(torch.bfloat16)
        self.x = x[off:].view(self.T, Hq + 2 * Hk, D)
        self.q, self.k, self.v = self.x[:, :Hq], self.x[:, Hq:Hq + Hk], self.x[:, Hq + Hk:]
        shape = (self.pages, page, Hk, D) if inside else (self.pages, Hk, page, D)
        self.cache = [torch.full(shape, 0x5A if mx else 3.25, dtype=torch.uint8 if mx else torch.bfloat16, device="cuda") for _ in range(2)]
        if inside:
            self.cache = [c.transpose(1, 2) for c in self.cache]
        self.units = [torch.full((self.pages, Hk, page, D // 32), 0x33, dtype=torch.uint8, device="cuda") if mx else None for _ in range(2)]
        self.w = [1 + 0.3 * rand(D) for _ in range(2)]
        self.q_out = torch.full((self.T, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")

    def batch(self, g):
        return g.kv_batch(self.T, torch.from_numpy(self.q_start).cuda(), torch.from_numpy(self.kv_len).cuda(), torch.from_numpy(self.table).cuda())

    def kv(self, g):
        return g.kv_cache(*self.cache, *self.units)


def check(g, b, rot, inter, norm=True, pos=None):
    Hq, Hk, D = b.q.shape[1], b.k.shape[1], b.q.shape[2]
    turns, frac = fractions(g, rot)
    f = g.qk_rope(b.T, Hq, Hk, D, rot, 0, layout=int(inter), norm=int(norm), eps=1e-5, amplitude=1.1, turns=turns, q=b.q, k=b.k, v=b.v, w_q=b.w[0] if norm else None,
                  w_k=b.w[1] if norm else None, q_out=b.q_out, pos=None if pos is None else torch.tensor(pos, dtype=torch.int32, device="cuda"))
    g.fp8_kv_append(f, b.kv(g), b.batch(g))
    torch.cuda.synchronize()
    at = heads.places(b.q_start, b.kv_len, b.T)
    theta = heads.angle([p for _, p in at] if pos is None else pos, frac)
    e = (D / 32 + 24) * 2.0 ** -24 * 1.1
    xs = [f64(t) for t in (b.q, b.k)]
    ns = [heads.norm(x, f64(w), 1e-5) if norm else x for x, w in zip(xs, b.w)]
    refs = [heads.rotate(n, theta, inter, 1.1) for n in ns] + [f64(b.v)]
    slack = [e * pairs_magnitude(n, rot, inter) for n in ns] + [np.zeros_like(refs[2])]
    q_out = f64(b.q_out)
    want = [np.full((b.pages, Hk, b.page, D), np.nan) for _ in range(2)]
    room = [np.zeros((b.pages, Hk, b.page, D)) for _ in range(2)]
    for t, (s, p) in enumerate(at):
        if s < 0:
            assert np.all(q_out[t] == 5.0)
            continue
        assert np.all(np.abs(q_out[t] - refs[0][t]) <= slack[0][t] + 2.0 ** -8 * np.abs(refs[0][t]) + 1e-38)
        if p < 0 or p >= b.table.shape[1] * b.page or not 0 <= b.table[s, p // b.page] < b.pages:
            continue
        for i in range(2):
            want[i][b.table[s, p // b.page], :, p % b.page] = refs[1 + i][t]
            room[i][b.table[s, p // b.page], :, p % b.page] = slack[1 + i][t]
    for i in range(2):
        raw = b.cache[i].cpu().numpy() if b.mx else f64(b.cache[i])
        kept = np.isnan(want[i])
        if not b.mx:
            assert np.all(raw[kept] == 3.25)
            assert np.all(np.abs(raw - want[i])[~kept] <= (room[i] + 2.0 ** -8 * np.abs(want[i]))[~kept] + 1e-38)
            continue
        units = b.units[i].cpu().numpy()
        assert np.all(raw[kept] == 0x5A) and np.all(units[kept[..., ::32]] == 0x33)
        ref = np.where(kept, 0, want[i])
        exp = heads.mx_exponents(ref)
        near = heads.mx_exponents(ref * (1 + 1e-5)) != heads.mx_exponents(ref * (1 - 1e-5))  # (a group's largest at a boundary)
        got = units.astype(int) - 127
        assert np.all((got == exp) | kept[..., ::32] | (near & (np.abs(got - exp) <= 1)))
        unit = np.repeat(np.exp2(exp + near), 32, axis=-1)
        err = np.abs(heads.mx_decode(raw, units) - ref)
        assert np.all((err <= room[i] + np.maximum(2.0 ** -4 * (np.abs(ref) + room[i]), 2.0 ** -10 * unit))[~kept])


CASES = [  # new, total, Hq, Hk, D, page, rot, interleaved
    ([1], [1], 1, 1, 64, 8, 64, False), ([1, 1, 1], [1, 16, 300], 32, 8, 128, 16, 128, False), ([5, 0, 33, 1], [5, 9, 64, 129], 6, 2, 128, 32, 64, True),
    ([130], [257], 3, 3, 64, 64, 32, False), ([3, 4], [40, 4], 4, 2, 96, 8, 96, False), ([3, 4], [40, 4], 2, 1, 256, 16, 256, True), ([7, 2], [7, 70], 5, 5, 32, 128, 16, False),
    ([2] * 70, list(range(2, 72)), 8, 4, 128, 16, 128, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}-{c[6]}")
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("inside", [False, True])
def test_append(g, case, mx, inside):
    new, total, Hq, Hk, D, page, rot, inter = case
    check(g, Batch(g, new, total, Hq, Hk, D, page, mx, inside), rot, inter)


@pytest.mark.parametrize("mx", [False, True])
def test_rows_of_single_elements(g, mx):
    check(g, Batch(g, [5, 9], [17, 9], 3, 2, 64, 16, mx, False, off=1), 64, False)
    check(g, Batch(g, [5, 9], [17, 9], 3, 2, 64, 16, mx, True, off=3), 20, True, norm=False)
    check(g, Batch(g, [5, 9], [17, 9], 3, 2, 128, 16, mx, True), 20, False)


def test_odd_head_in_bf16(g):
    check(g, Batch(g, [5, 9], [17, 9], 3, 2, 40, 16, False, False), 40, False)


@pytest.mark.parametrize("mx", [False, True])
def test_positions_of_its_own(g, mx):
    b = Batch(g, [5, 9], [17, 9], 3, 2, 64, 16, mx, False)
    check(g, b, 64, False, pos=[(1 << 31) - 1 - 1000 * t for t in range(b.T)])


@pytest.mark.parametrize("mx", [False, True])
def test_places_out_of_range(g, mx):
    """Positions below 0, behind the table, pages outside the cache, beginnings out of order: nothing is written but what has a place."""
    b = Batch(g, [6, 6, 6, 6], [6, 6, 40, 6], 4, 2, 64, 16, mx, False)
    b.kv_len[0] = 3                      # three tokens before the beginning
    b.kv_len[1] = b.table.shape[1] * 16 + 2
    b.table[1, :] = b.table[1, 0]
    b.table[2, 2] = b.pages              # positions 34 .. 39
    b.kv_len[3] = -5
    check(g, b, 64, False)
    b = Batch(g, [6, 6, 6], [6, 6, 40], 4, 2, 64, 16, mx, False)
    b.q_start[:] = [4, 6, 6, 1000]       # rows before the first sequence, an empty one, one that ends behind the rows
    b.kv_len[:] = [2, 9, 14]
    check(g, b, 64, False)


def test_unusual_values_in_8_bits(g):
    """Infinities saturate, a NaN makes its group NaN, zeros and the smallest values."""
    b = Batch(g, [6], [6], 1, 1, 64, 16, True, False, extra=0)
    v = b.x[:, 2]
    v[0, 3], v[1, 40], v[2], v[3], v[4, 0] = float("inf"), float("nan"), 0.0, 1e-38, -3.3e38
    v[5, :32], v[5, 32:] = 448.0, 450.0
    f = g.qk_rope(6, 1, 1, 64, 0, 0, q=b.q, k=b.k, v=b.v, q_out=b.q_out)
    g.fp8_kv_append(f, b.kv(g), b.batch(g))
    ref = f64(b.v)[:, 0]
    codes, units = (t[b.table[0, 0], 0, :6].cpu().numpy() for t in (b.cache[1], b.units[1]))
    assert np.array_equal(units.astype(int) - 127, heads.mx_exponents(ref))
    got = heads.mx_decode(codes, units)
    assert got[0, 3] == 448 * 2.0 ** 120 or got[0, 3] == 240 * 2.0 ** 120 or got[0, 3] == 256 * 2.0 ** 120
    assert np.all(np.isnan(got[1, 32:])) and np.all(np.isfinite(got[1, :32])) and not got[2].any() and units[1, 1] == 0xFF and not codes[1, 32:].any()
    fine = np.isfinite(ref) & ~np.isnan(got)
    unit = np.repeat(np.exp2(units.astype(float) - 127), 32, axis=-1)
    assert np.all((np.abs(got - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * unit))[fine])
