"""A run of the operators as a model uses them: a prompt in chunks and then single tokens, through the norm and rotation into the cache and
attention over it, beside attention over everything in 64 bits; eager and from a captured step."""
import numpy as np
import pytest
import torch

from oracle import heads
from test_gpu_qk_rope import f64, fractions

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import fp8_mixed_precision_saturating_gb300 as m
    return m


@pytest.mark.parametrize("mx", [False, True])
def test_chunks_then_tokens(g, mx):
    Hq, Hk, D, P = 8, 2, 64, 16
    lens, steps = [70, 33, 5], [64, 48, 1, 1, 1]  # what is there at the end; most new tokens of each call
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = [rand(n + 3, Hq + 2 * Hk, D).to(torch.bfloat16) for n in lens]
    w = [1 + 0.2 * rand(D) for _ in range(2)]
    turns, frac = fractions(g, D)
    pages = 32
    shape = (pages, Hk, P, D)
    cache = [torch.zeros(shape, dtype=torch.uint8 if mx else torch.bfloat16, device="cuda") for _ in range(2)]
    units = [torch.zeros(pages, Hk, P, D // 32, dtype=torch.uint8, device="cuda") if mx else None for _ in range(2)]
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[:24].view(3, 8).contiguous()
    kv = g.kv_cache(*cache, *units)
    have = [0, 0, 0]
    T = 130
    qkv, q_out, out = (torch.zeros(T, n, D, dtype=torch.bfloat16, device="cuda") for n in (Hq + 2 * Hk, Hq, Hq))
    start, kv_len = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    f = g.qk_rope(T, Hq, Hk, D, D, 0, norm=1, turns=turns, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:], w_q=w[0], w_k=w[1], q_out=q_out)
    a, b = g.paged_attention(Hq, D ** -0.5, q=q_out, out=out), g.kv_batch(T, start, kv_len, table)
    n = g.fp8_paged_attention_workspace_bytes(a, kv, b)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")

    def step():
        g.fp8_kv_append(f, kv, b)
        g.fp8_paged_attention(a, kv, b, ws, n)

    step()  # (nothing yet)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    got = [[] for _ in lens]
    for i, most in enumerate(steps):
        new = [min(most, m + 3 - h) if most > 1 else min(1, m + 3 - h) for m, h in zip(lens, have)]
        rows = torch.cat([xs[h:h + c] for xs, h, c in zip(x, have, new)])
        qkv[: rows.shape[0]] = rows
        have = [h + c for h, c in zip(have, new)]
        start.copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32))
        kv_len.copy_(torch.tensor(have, dtype=torch.int32))
        graph.replay() if i % 2 else step()
        torch.cuda.synchronize()
        at = 0
        for s, c in enumerate(new):
            got[s].append(f64(out[at:at + c]))
            at += c
    g.fp8_poll_device_error()
    for s in range(3):
        n = have[s]
        xs, theta = f64(x[s])[:n], heads.angle(range(n), frac)
        q = heads.forward(xs[:, :Hq], f64(w[0]), 1e-6, theta, False)
        k = heads.forward(xs[:, Hq:Hq + Hk], f64(w[1]), 1e-6, theta, False)
        page = lambda y: np.concatenate([y, np.zeros((-n % P, Hk, D))]).reshape(-1, P, Hk, D).transpose(0, 2, 1, 3)  # noqa: E731
        ref = heads.attention(q, page(k), page(xs[:, Hq + Hk:]), [0, n], [n], np.arange(-(-n // P))[None], D ** -0.5)[0]
        y = np.concatenate(got[s])
        assert y.shape == ref.shape
        # queries and outputs in bf16, the cache in bf16 or 8 bits (half a step 2^-4): scores move by that share of their spread, a few times sqrt(D)
        limit = 0.2 if mx else 0.02
        assert np.linalg.norm(y - ref) <= limit * np.linalg.norm(ref)
