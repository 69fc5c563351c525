"""Rotation, append and attention where their documentation allows what the other tests do not ask for: elements more than 2^31 from a
tensor's beginning, units cut into few and into many parts, pages of several sequences, output over the queries, calls at once and
captured ones, values of every 8-bit unit and infinities among the keys that all rows see. Bounds: as in the operators' own tests;
where the same numbers go through the same operations the results are the same bits."""
import os
import re

import numpy as np
import pytest
import torch

from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(*s, seed=0, dt=torch.bfloat16):
    return torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dt)


@pytest.mark.parametrize("mx", [False, True])
def test_a_cache_beyond_32_bits(g, mx):
    """The last pages of a cache of more than 2^31 elements (2^32 in 8 bits) against a cache of those pages alone."""
    D, page, H, Hq, new, total = 128, 4096, 2, 6, 37, 4096 + 300
    pages = (1 << (32 if mx else 31)) // (page * H * D) + 3
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("not enough memory")
    q, k, v = (randn(total, n, D, seed=n + i) for i, n in enumerate((Hq, H, H)))
    w = randn(D, seed=9, dt=torch.float32)
    turns = g.rope_turns(D, 10000.0)
    results = []
    for n, where in ((pages, (pages - 1, pages - 2)), (2, (1, 0))):
        kind = torch.uint8 if mx else torch.bfloat16
        cache = [torch.empty(n, H, page, D, dtype=kind, device="cuda") for _ in range(2)]
        units = [torch.empty(n, H, page, D // 32, dtype=torch.uint8, device="cuda") for _ in range(2)] if mx else [None, None]
        c, table = g.kv_cache(*cache, *units), i32(*where).view(1, 2)
        out, lse, q_out = torch.empty_like(q[:new]), torch.empty(new, Hq, device="cuda"), torch.empty_like(q)
        f = g.qk_rope(total, Hq, H, D, D, g.FP8_DT_BF16, norm=g.FP8_NORM_RMS, turns=turns, q=q, k=k, v=v, w_k=w, q_out=q_out)
        g.fp8_kv_append(f, c, g.kv_batch(total, i32(0, total), i32(total), table))
        b = g.kv_batch(new, i32(0, new), i32(total), table)
        a = g.paged_attention(Hq, D ** -0.5, q=q_out[-new:], out=out, lse=lse)
        size = g.fp8_paged_attention_workspace_bytes(a, c, b)
        g.fp8_paged_attention(a, c, b, torch.zeros(size, dtype=torch.uint8, device="cuda"), size)
        at = [x[p, :, :r].clone() for x in cache + ([] if not mx else units) for p, r in zip(where, (page, total - page))]
        results.append([out, lse, q_out] + at)
        torch.cuda.synchronize()
        del c, cache, units
        torch.cuda.empty_cache()
    g.fp8_poll_device_error()
    assert torch.isfinite(results[0][1]).all()
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_heads_beyond_32_bits(g):
    """Three tokens 2^30 elements and more apart: rotation, gradient, append's inputs and attention's, against the same next to each other."""
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("not enough memory")
    D, Hq, Hk, T, ld = 64, 4, 2, 3, (1 << 30) + 64
    n = Hq + 2 * Hk
    x, dy = randn(T, n, D, seed=1), randn(T, n, D, seed=2)
    big, big_out = (torch.empty(2 * ld + n * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far, far_out = (t.as_strided((T, n, D), (ld, D, 1)) for t in (big, big_out))
    turns, w = g.rope_turns(D, 10000.0), randn(D, seed=3, dt=torch.float32)
    got = []
    for x_, y_ in ((x, torch.empty_like(x)), (far, far_out)):
        x_.copy_(x)
        f = g.qk_rope(T, Hq, Hk, D, D, g.FP8_DT_BF16, norm=g.FP8_NORM_RMS, turns=turns, q=x_[:, :Hq], k=x_[:, Hq:Hq + Hk], w_q=w, w_k=w, q_out=y_[:, :Hq], k_out=y_[:, Hq:Hq + Hk])
        g.fp8_qk_rope_fwd(f)
        fwd = y_[:, : Hq + Hk].clone()
        y_.copy_(dy)
        dw = [torch.empty(D, device="cuda") for _ in range(2)]
        back = g.qk_rope_grad(dq_out=y_[:, :Hq], dk_out=y_[:, Hq:Hq + Hk], dq=y_[:, :Hq], dk=y_[:, Hq:Hq + Hk], dw_q=dw[0], dw_k=dw[1])
        size = g.fp8_qk_rope_bwd_workspace_bytes(f, back)
        g.fp8_qk_rope_bwd(f, back, torch.empty(size, dtype=torch.uint8, device="cuda"), size)
        bwd = y_[:, : Hq + Hk].clone()
        cache = [torch.zeros(1, Hk, 8, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        c, b = g.kv_cache(*cache), g.kv_batch(T, i32(0, T), i32(T), i32(0).view(1, 1))
        f = g.qk_rope(T, Hq, Hk, D, D, g.FP8_DT_BF16, turns=turns, q=x_[:, :Hq], k=x_[:, Hq:Hq + Hk], v=x_[:, Hq + Hk:], q_out=y_[:, :Hq])
        g.fp8_kv_append(f, c, b)
        a = g.paged_attention(Hq, 0.125, q=y_[:, :Hq], out=y_[:, Hq:])
        size = g.fp8_paged_attention_workspace_bytes(a, c, b)
        g.fp8_paged_attention(a, c, b, torch.zeros(size, dtype=torch.uint8, device="cuda"), size)
        got.append([fwd, bwd, *dw, *cache, y_.clone()])
    torch.cuda.synchronize()
    g.fp8_poll_device_error()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new, total, heads_", [
    ([1], [40000], (1, 1)), ([1], [40000], (5, 1)), ([3], [40000], (8, 1)), ([1], [40000], (128, 1)), ([2], [21000], (64, 1)), ([12], [9000], (8, 1)),  # one unit over all CTAs
    ([4], [3000], (16, 2)), ([33], [1500], (8, 2)), ([64, 1, 7], [700, 3000, 130], (4, 4)),                                                            # few parts of full tiles
    ([9] * 40, [700 + 13 * i for i in range(40)], (12, 4)), ([40] * 24, [300 + 41 * i for i in range(24)], (4, 2)), ([100] * 12, [600] * 12, (6, 6))], ids=str)  # many units
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mx", [False, True])
def test_cut_units(g, new, total, heads_, D, mx):
    c = Case(g, new, total, *heads_, D, 64, mx, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("new, total, heads_", [([1] * 5, [100, 900, 4000, 1, 33], (8, 2)), ([70, 1], [3000, 500], (8, 2)), ([300], [300], (6, 3)), ([50], [20000], (4, 1))], ids=str)
def test_output_over_the_queries(g, new, total, heads_):
    c = Case(g, new, total, *heads_, 128, 16, extra=0)
    c.run()
    a, cc, b, ws, n = c.plans()
    x = c.q.clone()
    g.fp8_paged_attention(g.paged_attention(heads_[0], c.scale, q=x, out=x), cc, b, ws, n)
    assert torch.equal(x, c.out)


def test_sequences_that_share_pages(g):
    """A prefix in the pages of three sequences, and one page twice in a table."""
    for mx in (False, True):
        c = Case(g, [1, 5, 130], [300, 400, 530], 8, 2, 128, 32, mx)
        c.table[1, :8] = c.table[0, :8]
        c.table[2, :8] = c.table[0, :8]
        c.table[2, 9] = c.table[2, 10]
        c.run()
        c.check()


def test_unusual_values_that_all_rows_see(g):
    for new, total in (([1], [700]), ([40], [700]), ([300], [700])):
        for value in (float("inf"), float("nan")):
            for which in (0, 1):
                c = Case(g, new, total, 4, 2, 128, 16, seed=6)
                c.put(int(c.table[0, 20]), slice(3, 4), value, which=(which,), dims=slice(32, 33))
                c.run()
                c.check()


@pytest.mark.parametrize("new, total", [([1], [700]), ([40], [700]), ([130], [300])], ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_8_bit_units_of_every_size(g, new, total, D):
    """Values from 2^-127 units to ones that are infinite in bf16, keys with large and small units that cancel in the scale."""
    c = Case(g, new, total, 4, 2, D, 16, mx=True, scale=2.0 ** -40)
    for j, unit in ((0, 0), (5, 1), (40, 134), (41, 135), (77, 200), (128, 230), (300 - 131, 246)):
        c.units[1][int(c.table[0, j // 16]), :, j % 16, 0] = unit
    for j, unit in ((1, 0), (33, 135), (150, 140)):
        c.units[0][int(c.table[0, j // 16]), :, j % 16] = unit
    c.run()
    c.check()


def test_calls_at_once_and_captured_ones(g):
    """Rotation, its gradient, append and attention of two layers on two streams at once, from graphs with workspaces of their own, replayed
    with other inputs: the bits of single calls."""
    D, Hq, Hk, T, page, total = 128, 8, 2, 70, 16, 500

    class Layer:
        def __init__(self, seed):
            self.x, self.y, self.dx = (randn(T, Hq + 2 * Hk, D, seed=seed) for _ in range(3))
            self.w, self.dw = randn(2, D, seed=seed, dt=torch.float32), torch.empty(2, D, device="cuda")
            self.cache = [randn(40, Hk, page, D, seed=seed + i) for i in (1, 2)]
            self.out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
            parts = dict(q=self.x[:, :Hq], k=self.x[:, Hq:Hq + Hk], w_q=self.w[0], w_k=self.w[1], q_out=self.y[:, :Hq])
            common = (T, Hq, Hk, D, D, g.FP8_DT_BF16)
            turns = g.rope_turns(D, 10000.0)
            self.rope = g.qk_rope(*common, norm=g.FP8_NORM_RMS, turns=turns, k_out=self.y[:, Hq:Hq + Hk], **parts)
            self.append = g.qk_rope(*common, norm=g.FP8_NORM_RMS, turns=turns, v=self.x[:, Hq + Hk:], **parts)
            self.back = g.qk_rope_grad(dq_out=self.y[:, :Hq], dk_out=self.y[:, Hq:Hq + Hk], dq=self.dx[:, :Hq], dk=self.dx[:, Hq:Hq + Hk], dw_q=self.dw[0], dw_k=self.dw[1])
            self.lens = i32(total)
            self.c, self.b = g.kv_cache(*self.cache), g.kv_batch(T, i32(0, T), self.lens, torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40))
            self.a = g.paged_attention(Hq, D ** -0.5, q=self.y[:, :Hq], out=self.out)
            n = g.fp8_qk_rope_bwd_workspace_bytes(self.rope, self.back), g.fp8_paged_attention_workspace_bytes(self.a, self.c, self.b)
            self.ws = [(torch.zeros(i, dtype=torch.uint8, device="cuda"), i) for i in n]

        def run(self, stream=None):
            g.fp8_qk_rope_fwd(self.rope, stream=stream)
            g.fp8_qk_rope_bwd(self.rope, self.back, *self.ws[0], stream=stream)
            g.fp8_kv_append(self.append, self.c, self.b, stream=stream)
            g.fp8_paged_attention(self.a, self.c, self.b, *self.ws[1], stream=stream)

        def results(self):
            return [t.clone() for t in (self.out, self.y[:, : Hq + Hk], self.dx[:, : Hq + Hk], self.dw, *self.cache)]

    layers = [Layer(10), Layer(20)]
    graphs, streams = [], [torch.cuda.Stream() for _ in layers]
    for la in layers:
        la.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            la.run()
    for turn, length in enumerate((500, 333, 70)):
        for i, la in enumerate(layers):
            la.x.copy_(randn(T, Hq + 2 * Hk, D, seed=100 + 2 * turn + i))
            la.lens.fill_(length)
        torch.cuda.synchronize()
        want = []
        for la in layers:
            la.run()
            torch.cuda.synchronize()
            want.append(la.results())
        for way in ("streams", "graphs"):
            for la in layers:
                la.out.fill_(9.0)
                la.dw.fill_(9.0)
            torch.cuda.synchronize()
            for _ in range(4):
                for la, graph, s in zip(layers, graphs, streams):
                    if way == "streams":
                        la.run(s)
                    else:
                        with torch.cuda.stream(s):
                            graph.replay()
            torch.cuda.synchronize()
            for la, w in zip(layers, want):
                for x, y in zip(la.results(), w):
                    assert torch.equal(x, y), way
    g.fp8_poll_device_error()


def test_the_usage_example_runs():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    block = next(b for b in re.findall(r"```python\n(.*?)```", open(path).read(), re.S) if "fp8_kv_append" in b)
    import fp8_mixed_precision_saturating_gb300 as m
    env = {"torch": torch, "g": m}
    torch.manual_seed(0)
    exec(compile(block, "README.md", "exec"), env)
    torch.cuda.synchronize()
    m.fp8_poll_device_error()
    # a sequence of one token sees itself alone; one of zeros and a new token the new token's part of its values
    new = env["qkv"][:, 40:].repeat_interleave(4, dim=1)
    assert torch.equal(env["o"][2], new[2])
    o, v = env["o"].float(), new.float()
    share = (o * v).sum(-1) / (v * v).sum(-1)
    assert torch.all((share > 0) & (share <= 1.01)) and torch.allclose(o, share[..., None] * v, atol=0.05)
