"""Attention over a paged cache against the oracle in 64 bits: single tokens and chunks, ragged batches, groups of heads that do and do
not divide a tile, windows, both formats and layouts, pages of every size, rows that see nothing, unusual values in masked places.

Bounds. A score is a sum of D exact products in fp32: below (D + 8) 2^-24 of scale sum |q k| = big, in whatever order; the weight
adds the exponential's and the scale's own error, 2^-20 relative with its argument's rounding (2^-24 of at most 2^4 big): s = (D + 40) 2^-24 big + 2^-20 in all. The weights are
rounded to bf16 (half a step, 2^-8) for the product with the values, whose fp32 sums are below 2^-20 of the magnitudes for these lengths;
out adds its own half step. So |out - ref| <= (2^-8 + 2 s + 2^-20) sum w |v| / sum w + 2^-8 |ref|, |lse - ref| <= 2 s + 2^-20 (1 + |ref|)."""
import numpy as np
import pytest
import torch

from oracle import heads
from test_gpu_qk_rope import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


class Case:
    def __init__(self, g, new, total, Hq, Hk, D, page, mx=False, inside=False, window=0, extra=3, seed=0, size=1.0, scale=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.g, self.D, self.page, self.mx, self.window, self.Hq, self.Hk = g, D, page, mx, window, Hq, Hk
        self.scale = D ** -0.5 if scale is None else scale
        self.T = sum(new) + extra
        need = [-(-t // page) for t in total]
        self.pages, width = sum(need) + 2, max(need) + 1
        order = torch.randperm(self.pages, generator=gen, device="cuda").cpu().tolist()
        self.table = np.full((len(new), width), 1 << 30, dtype=np.int32)
        for s, n in enumerate(need):
            self.table[s, :n] = [order.pop() for _ in range(n)]
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.array(total, dtype=np.int32)
        self.q = (size * rand(self.T, Hq, D)).to(torch.bfloat16)
        shape = (self.pages, page, Hk, D) if inside else (self.pages, Hk, page, D)
        self.units = [None, None]
        self.cache = []
        for i in range(2):
            if mx:
                codes = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
                codes[(codes & 127) == 127] = 0
                self.units[i] = torch.randint(118, 121, (self.pages, Hk, page, D // 32), generator=gen, device="cuda", dtype=torch.uint8)
                self.cache.append(codes)
            else:
                self.cache.append(rand(*shape).to(torch.bfloat16))
        if inside:
            self.cache = [c.transpose(1, 2) for c in self.cache]
        self.out = torch.full((self.T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, Hq), 9.0, device="cuda")
        self.spoil(need)

    def spoil(self, need):
        """NaN behind every sequence's end: in the rest of its last page, and in pages of nobody."""
        mine = set()
        for s, n in enumerate(need):
            mine |= set(self.table[s, :n].tolist())
            if n and self.kv_len[s] % self.page:
                self.put(int(self.table[s, n - 1]), slice(int(self.kv_len[s]) % self.page, None), float("nan"))
        for p in set(range(self.pages)) - mine:
            self.put(p, slice(None), float("nan"))

    def put(self, page, rows, value, which=(0, 1), dims=slice(None)):
        for i in which:
            if self.mx:
                if np.isnan(value):
                    self.units[i][page, :, rows] = 0xFF
                else:
                    self.cache[i][page, :, rows, dims] = 0x7E if value > 0 else 0xFE
            else:
                self.cache[i][page, :, rows, dims] = value

    def plans(self):
        g = self.g
        a = g.paged_attention(self.Hq, self.scale, window=self.window, q=self.q, out=self.out, lse=self.lse)
        self.dev = [torch.from_numpy(x).cuda() for x in (self.q_start, self.kv_len, self.table)]
        c, b = g.kv_cache(*self.cache, *self.units), g.kv_batch(self.T, *self.dev)
        n = g.fp8_paged_attention_workspace_bytes(a, c, b)
        return a, c, b, torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"), n

    def run(self, plans=None):
        self.g.fp8_paged_attention(*(plans or self.plans()))
        torch.cuda.synchronize()
        self.g.fp8_poll_device_error()

    def values(self):
        if not self.mx:
            return [f64(c) for c in self.cache]
        return [heads.mx_decode(c.cpu().numpy(), u.cpu().numpy()) for c, u in zip(self.cache, self.units)]

    def check(self):
        k, v = self.values()
        out, lse, mag, big = heads.attention(f64(self.q), k, v, self.q_start, self.kv_len, self.table, self.scale, self.window)
        got, got_lse = f64(self.out), f64(self.lse)
        nobody = np.array([s < 0 for s, _ in heads.places(self.q_start, self.kv_len, self.T)])
        assert np.all(got[nobody] == 9.0) and np.all(got_lse[nobody] == 9.0)
        out, lse, mag, big, got, got_lse = (x[~nobody] for x in (out, lse, mag, big, got, got_lse))
        s = (self.D + 40) * 2.0 ** -24 * big + 2.0 ** -20
        fine = np.isfinite(out)
        with np.errstate(invalid="ignore"):
            bad = np.abs(got - out) > (2.0 ** -8 + 2 * s[..., None] + 2.0 ** -20) * mag + 2.0 ** -8 * np.abs(out)
        assert not np.any(bad & fine), (np.argwhere(bad & fine)[:4], np.abs(got - out)[bad & fine][:4])
        assert np.array_equal(np.isnan(got), np.isnan(out)) and np.array_equal(got[np.isinf(out)], out[np.isinf(out)])
        fine = np.isfinite(lse)
        assert np.all(np.abs(got_lse - lse)[fine] <= (2 * s + 2.0 ** -20 * (1 + np.abs(lse)))[fine])
        assert np.array_equal(np.isnan(got_lse), np.isnan(lse)) and np.array_equal(got_lse == -np.inf, lse == -np.inf)


SHAPES = [  # new, total
    ([1], [1]), ([1], [300]), ([1, 1, 1, 1], [1, 128, 129, 517]), ([5, 0, 33, 1], [5, 9, 164, 1029]), ([130], [130]), ([300, 2], [700, 2]), ([3], [4096]), ([1] * 37, list(range(1, 371, 10))),
]


@pytest.mark.parametrize("new, total", SHAPES, ids=str)
@pytest.mark.parametrize("heads_", [(1, 1), (8, 2), (6, 2), (5, 1), (32, 8), (128, 1)], ids=str)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mx", [False, True])
def test_attention(g, new, total, heads_, D, mx):
    if sum(new) * heads_[0] * max(total) > 4e6:
        pytest.skip("the oracle's time")
    c = Case(g, new, total, *heads_, D, 16, mx, seed=len(new))
    c.run()
    c.check()


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 4096])
@pytest.mark.parametrize("inside", [False, True])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_pages(g, page, inside, mx, D):
    c = Case(g, [1, 40, 3], [333, 40, 700], 4, 2, D, page, mx, inside)
    c.run()
    c.check()


@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 1000])
@pytest.mark.parametrize("mx", [False, True])
def test_windows(g, window, mx):
    c = Case(g, [1, 150, 3], [333, 150, 700], 6, 2, 64, 32, mx, window=window)
    c.run()
    c.check()


def test_long_contexts_are_split(g):
    for mx in (False, True):
        c = Case(g, [1, 2], [30011, 17], 8, 2, 128, 64, mx)
        c.run()
        c.check()
    c = Case(g, [40], [9000], 8, 1, 64, 64)
    c.run()
    c.check()


def test_scores_of_every_size(g):
    """Peaked weights, scores that grow or fall along the keys (the running maximum moves at every tile), tiny and negative scales."""
    for size, scale in ((8.0, None), (1.0, 1e-30), (1.0, -0.3), (1.0, 0.0), (30.0, 1.0)):
        c = Case(g, [2, 140], [900, 500], 4, 2, 64, 16, size=size, scale=scale)
        c.run()
        c.check()
    for sign in (1, -1):
        c = Case(g, [1, 140], [900, 500], 4, 2, 64, 16)
        c.q[:] = 1.0
        for s in range(2):
            for j in range(int(c.kv_len[s])):
                c.cache[0][int(c.table[s, j // 16]), :, j % 16] = sign * j * 0.05
        c.run()
        c.check()


def test_rows_that_see_nothing(g):
    """More new tokens than the cache holds, empty caches, no new tokens, rows of nobody at both ends, beginnings out of order."""
    c = Case(g, [20, 5, 0, 7], [20, 5, 64, 7], 4, 2, 128, 16)
    c.kv_len[:] = [13, 0, 64, -3]
    c.run()
    c.check()
    assert torch.all(c.out[:7] == 0) and torch.all(c.lse[:7] == -np.inf)
    c = Case(g, [20, 5, 9], [40, 5, 30], 4, 2, 128, 16, mx=True)
    c.q_start[:] = [3, 20, 20, 1000]
    c.run()
    c.check()
    c = Case(g, [20, 5], [40, 5], 4, 2, 128, 16)
    c.kv_len[0] = 10 ** 6  # the table ends before
    c.run()
    c.check()


def test_pages_outside_the_cache_hold_zeros(g):
    for mx in (False, True):
        c = Case(g, [3, 1], [200, 90], 4, 2, 64, 16, mx)
        c.table[0, 2], c.table[0, 7], c.table[1, 0] = -1, c.pages, 1 << 30
        c.run()
        c.check()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("which", [0, 1])
def test_later_tokens_do_not_reach_back(g, mx, which):
    """What is not finite in a key or value that a row does not see leaves the row as it was; the rows that see it get it."""
    for new, total in (([150], [150]), ([9, 1], [140, 33])):
        for value in (float("nan"),) if mx else (float("nan"), float("inf"), -float("inf")):
            c = Case(g, new, total, 4, 2, 128, 16, mx, seed=4)
            c.run()
            clean = c.out.clone()
            at = total[0] - 5
            c.put(int(c.table[0, at // 16]), slice(at % 16, at % 16 + 1), value, which=(which,), dims=slice(64, 96))
            c.run()
            c.check()
            assert torch.equal(c.out[: new[0] - 5], clean[: new[0] - 5])


def test_windows_keep_out_what_is_not_finite(g):
    for mx in (False, True):
        c = Case(g, [40], [300], 4, 2, 64, 16, mx, window=100)
        for j in (10, 170, 190):  # behind every window, behind some
            c.put(int(c.table[0, j // 16]), slice(j % 16, j % 16 + 1), float("nan"), which=(1,))
        c.run()
        c.check()


def test_strides_and_no_lse(g):
    c = Case(g, [5, 30], [70, 30], 8, 2, 64, 16)
    c.run()
    wide = torch.full((8, c.T, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(8, c.T, 80, dtype=torch.bfloat16, device="cuda")
    q[..., 8:72] = c.q.transpose(0, 1)
    a, cc, b, ws, n = c.plans()
    other = g.paged_attention(8, c.scale, q=q.transpose(0, 1)[..., 8:72], out=wide.transpose(0, 1)[..., :64])
    g.fp8_paged_attention(other, cc, b, ws, n)
    assert torch.equal(wide.transpose(0, 1)[..., :64], c.out) and torch.all(wide[..., 64:] == 9.0)


def test_the_same_bits_and_workspaces(g):
    """Twice the same; with a workspace that other calls have used; on two streams at once with their own."""
    cases = [Case(g, [1] * 9, [100 + 301 * i for i in range(9)], 8, 2, 128, 16, seed=1), Case(g, [200, 1], [900, 5000], 8, 2, 128, 16, seed=2), Case(g, [1], [20000], 8, 2, 128, 64, True, seed=3)]
    plans = [c.plans() for c in cases]
    most = max(plans, key=lambda p: p[4])
    want = []
    for c, p in zip(cases, plans):
        c.run(p)
        want.append((c.out.clone(), c.lse.clone()))
        c.check()
    for _ in range(3):
        for c, p, w in zip(cases, plans, want):
            c.out.fill_(9.0)
            c.run((*p[:3], most[3], most[4]))
            assert torch.equal(c.out, w[0]) and torch.equal(c.lse, w[1])
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.out.fill_(9.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(plans, streams):
            g.fp8_paged_attention(*p, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w[0]) and torch.equal(c.lse, w[1])


def test_a_captured_call_serves_other_lengths(g):
    c = Case(g, [1, 1, 1], [700, 300, 40], 8, 2, 128, 16)
    p = c.plans()
    c.run(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.fp8_paged_attention(*p)
    for lens in ([1, 300, 39], [700, 0, 17], [512, 129, 1]):
        c.kv_len[:] = lens
        c.dev[1].copy_(torch.from_numpy(c.kv_len))
        c.out.fill_(9.0)
        c.lse.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
