"""Refusals of the heads', cache's and attention's entry points, on CPU: every call below is refused before it touches the GPU, the same
way through both bindings. Device addresses are made-up numbers; nothing is dereferenced."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("host-side checks only: made-up device addresses", allow_module_level=True)

A, B, C, S, ODD = 0x10000, 0x20000, 0x30000, 0x40000, 0x10001


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    try:
        __graft_entry__._build_module().build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as m
    return m


def refused(g, status, what, name, *args):
    for fn in {getattr(g, name), getattr(g, "_by_ctypes", {}).get(name, getattr(g, name))}:
        with pytest.raises(g.Fp8Error) as e:
            fn(*args)
        assert e.value.status == status and what in str(e.value), str(e.value)


def rope(g, **kw):
    """Heads that a call would take; what is wrong comes in by name."""
    a = dict(tokens=4, q_heads=2, k_heads=1, head_dim=64, rot_dims=64, dt=0, layout=0, norm=1, eps=1e-6, amplitude=1.0, turns=S, q=A, ld_q=192, hs_q=64, k=A + 256, ld_k=192,
             hs_k=64, q_out=B, ld_q_out=128, hs_q_out=64, k_out=C, ld_k_out=64, hs_k_out=64)
    a.update(kw)
    first = [a.pop(n) for n in ("tokens", "q_heads", "k_heads", "head_dim", "rot_dims", "dt")]
    return g.qk_rope(*first, **a)


BAD_ROPE = [("negative", dict(tokens=-1)), ("negative", dict(q_heads=-1)), ("negative", dict(head_dim=0, rot_dims=0)), ("type", dict(dt=2)), ("layout", dict(layout=2)),
            ("norm", dict(norm=3)), ("rot_dims", dict(rot_dims=3)), ("rot_dims", dict(rot_dims=66)), ("rot_dims", dict(rot_dims=-2)), ("eps", dict(eps=-1.0)),
            ("eps", dict(eps=math.nan)), ("eps", dict(eps=math.inf)), ("amplitude", dict(amplitude=0.0)), ("amplitude", dict(amplitude=math.inf)), ("turns", dict(turns=None)),
            ("without a norm", dict(norm=0, w_k=S)), ("overlap", dict(ld_q=64)), ("overlap", dict(hs_q_out=32)), ("overlap", dict(ld_k=0)), ("overlap", dict(ld_k=-64)),
            ("in place", dict(q_out=A)), ("in place", dict(k_out=A + 256))]


def test_rope(g):
    for what, kw in BAD_ROPE:
        refused(g, g.FP8_ERR_INVALID_ARG, what, "fp8_qk_rope_fwd", rope(g, **kw))
    for what, kw in (("layer", dict(norm=2)), ("tokens", dict(tokens=1 << 31)), ("heads", dict(k_heads=32768, hs_k=64, ld_k=1 << 22, ld_k_out=1 << 22)), ("head_dim", dict(head_dim=257))):
        refused(g, g.FP8_ERR_UNSUPPORTED, what, "fp8_qk_rope_fwd", rope(g, **kw))
    for kw in (dict(turns=S + 4), dict(pos=S + 2), dict(w_q=S + 2), dict(q=ODD), dict(dt=1, k_out=C + 2)):
        refused(g, g.FP8_ERR_ALIGNMENT, "aligned", "fp8_qk_rope_fwd", rope(g, **kw))
    refused(g, g.FP8_ERR_INVALID_ARG, "null arguments", "fp8_qk_rope_fwd", None)
    refused(g, g.FP8_ERR_INVALID_ARG, "without", "fp8_qk_rope_fwd", rope(g, q_out=None))
    refused(g, g.FP8_ERR_INVALID_ARG, "without", "fp8_qk_rope_fwd", rope(g, k=None))
    refused(g, g.FP8_ERR_INVALID_ARG, "no output", "fp8_qk_rope_fwd", rope(g, q=None, k=None, q_out=None, k_out=None))
    assert g.fp8_qk_rope_fwd(rope(g, tokens=0)) == 0
    # heads apart, tokens inside: the other nesting
    refused(g, g.FP8_ERR_INVALID_ARG, "overlap", "fp8_qk_rope_fwd", rope(g, ld_q=64, hs_q=255))


def test_rope_backward(g):
    ws = 1 << 20
    def grad(**kw):
        return g.qk_rope_grad(**{**dict(dq_out=A, ld_dq_out=128, hs_dq_out=64, dk_out=B, ld_dk_out=64, hs_dk_out=64, dq=C, ld_dq=128, hs_dq=64, dk=S, ld_dk=64, hs_dk=64), **kw})
    call = "fp8_qk_rope_bwd"
    inv = g.FP8_ERR_INVALID_ARG
    for what, kw in BAD_ROPE[:16]:
        refused(g, inv, what, call, rope(g, **kw), grad(), S, ws)
    refused(g, inv, "null gradients", call, rope(g), None, S, ws)
    refused(g, inv, "without a norm", call, rope(g, norm=0), grad(dw_q=S), S, ws)
    refused(g, inv, "overlap", call, rope(g), grad(ld_dq=64), S, ws)
    refused(g, inv, "in place", call, rope(g), grad(dq=A, ld_dq=192), S, ws)
    refused(g, inv, "needs k", call, rope(g, k=None), grad(), S, ws)
    refused(g, inv, "without dk_out", call, rope(g), grad(dk_out=None), S, ws)
    refused(g, inv, "no output", call, rope(g), grad(dq=None, dk=None), S, ws)
    refused(g, inv, "needed", call, rope(g), grad(dw_k=S), None, 0)
    refused(g, inv, "needed", call, rope(g), grad(dw_k=S), A, 64)
    refused(g, inv, "negative workspace", call, rope(g), grad(dw_k=S), A, -1)
    refused(g, g.FP8_ERR_ALIGNMENT, "workspace", call, rope(g), grad(dw_k=S), A + 8, ws)
    refused(g, g.FP8_ERR_ALIGNMENT, "aligned", call, rope(g), grad(dq=ODD), S, ws)
    refused(g, g.FP8_ERR_ALIGNMENT, "aligned", call, rope(g), grad(dw_q=S + 2), S, ws)
    assert g.fp8_qk_rope_bwd_workspace_bytes(rope(g), grad()) == 0 and g.fp8_qk_rope_bwd_workspace_bytes(rope(g), grad(dw_q=S)) > 0
    for f, b in ((rope(g, dt=7), grad()), (rope(g), None), (rope(g, norm=0), grad(dw_q=S))):
        with pytest.raises(g.Fp8Error):
            g.fp8_qk_rope_bwd_workspace_bytes(f, b)


def cache(g, **kw):
    a = dict(k=A, v=B, k_scale=0, v_scale=0, format=0, pages=9, page_size=16, heads=1, head_dim=64, page_stride=1024, head_stride=1024, token_stride=64)
    a.update(kw)
    return g.fp8_kv_cache_t(**a)


def batch(g, **kw):
    a = dict(tokens=4, seqs=2, table_width=3, ld_table=3, q_start=S, kv_len=S, page_table=S)
    a.update(kw)
    return g.fp8_kv_batch_t(**a)


MX = dict(format=1, k_scale=C, v_scale=C)
INVALID_CACHE = [("format", dict(format=2)), ("size", dict(pages=-1)), ("size", dict(heads=0)), ("size", dict(head_dim=0)), ("size", dict(page_size=0)),
                 ("null cache buffers", dict(k=0)), ("needs its scales", dict(format=1)), ("needs its scales", dict(MX, v_scale=0)), ("has no scales", dict(k_scale=C)),
                 ("overlap", dict(token_stride=32)), ("overlap", dict(page_stride=1016)), ("overlap", dict(heads=2)), ("overlap", dict(token_stride=-64))]
UNSUPPORTED_CACHE = [("page_size", dict(page_size=4)), ("page_size", dict(page_size=24)), ("page_size", dict(page_size=8192)), ("2^40", dict(page_stride=1 << 41)),
                     ("head_dim", dict(head_dim=264, token_stride=264, head_stride=1 << 20, page_stride=1 << 20)), ("% 32", dict(MX, head_dim=48))]
UNALIGNED_CACHE = [dict(k=A + 8), dict(v=B + 2), dict(token_stride=68, page_stride=2048), dict(page_stride=1028), dict(MX, k_scale=C + 4), dict(MX, page_stride=1032)]
INVALID_BATCH = [("size", dict(tokens=-1)), ("size", dict(seqs=-1)), ("size", dict(table_width=-1)), ("null", dict(q_start=0)), ("null", dict(kv_len=0)), ("null", dict(page_table=0)),
                 ("ld_table", dict(ld_table=2))]


def each_bad_cache_and_batch(g, call):
    inv, un, al = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_UNSUPPORTED, g.FP8_ERR_ALIGNMENT
    for what, kw in INVALID_CACHE:
        call(inv, what, cache(g, **kw), batch(g))
    for what, kw in UNSUPPORTED_CACHE:
        call(un, what, cache(g, **kw), batch(g))
    for kw in UNALIGNED_CACHE:
        call(al, "16 bytes", cache(g, **kw), batch(g))
    for what, kw in INVALID_BATCH:
        call(inv, what, cache(g), batch(g, **kw))
    for kw in (dict(q_start=S + 2), dict(kv_len=S + 1), dict(page_table=S + 2)):
        call(al, "aligned", cache(g), batch(g, **kw))
    call(un, "2^31", cache(g), batch(g, tokens=1 << 31))
    call(inv, "null cache", None, batch(g))
    call(inv, "null batch", cache(g), None)


def test_append(g):
    def heads(**kw):
        return rope(g, **{**dict(v=C, ld_v=64, hs_v=64, k_out=None), **kw})
    name = "fp8_kv_append"
    inv = g.FP8_ERR_INVALID_ARG
    each_bad_cache_and_batch(g, lambda status, what, c, b: refused(g, status, what, name, heads(), c, b))
    for what, kw in BAD_ROPE[:16]:
        if "k_out" not in kw:
            refused(g, inv, what, name, heads(**kw), cache(g), batch(g))
    refused(g, g.FP8_ERR_UNSUPPORTED, "bf16", name, heads(dt=1), cache(g), batch(g))
    refused(g, inv, "into a cache", name, heads(), cache(g, heads=2, head_stride=1024, page_stride=2048), batch(g))
    refused(g, inv, "into a cache", name, heads(head_dim=32, rot_dims=32), cache(g), batch(g))
    refused(g, inv, "in the batch", name, heads(), cache(g), batch(g, tokens=3))
    refused(g, inv, "k_out", name, heads(k_out=C), cache(g), batch(g))
    refused(g, inv, "null k or v", name, heads(v=None), cache(g), batch(g))
    refused(g, inv, "q without q_out", name, heads(q_out=None), cache(g), batch(g))
    refused(g, inv, "overlap", name, heads(ld_v=32), cache(g), batch(g))
    assert g.fp8_kv_append(heads(tokens=0), cache(g), batch(g, tokens=0)) == 0 and g.fp8_kv_append(heads(), cache(g), batch(g, seqs=0, q_start=0)) == 0


def test_attention(g):
    def attn(**kw):
        a = dict(q_heads=4, scale=0.125, window=0, q=A, ld_q=256, hs_q=64, out=B, ld_out=256, hs_out=64)
        a.update(kw)
        return g.paged_attention(a.pop("q_heads"), a.pop("scale"), **a)
    name, ws = "fp8_paged_attention", (S, 1 << 40)
    inv, un, al = g.FP8_ERR_INVALID_ARG, g.FP8_ERR_UNSUPPORTED, g.FP8_ERR_ALIGNMENT
    each_bad_cache_and_batch(g, lambda status, what, c, b: refused(g, status, what, name, attn(), c, b, *ws))
    for what, kw in (("no query heads", dict(q_heads=0)), ("window", dict(window=-1)), ("scale", dict(scale=math.inf)), ("scale", dict(scale=math.nan)), ("null q", dict(q=None)),
                     ("null q", dict(out=None)), ("overlap", dict(ld_q=64)), ("overlap", dict(hs_out=32))):
        refused(g, inv, what, name, attn(**kw), cache(g), batch(g), *ws)
    refused(g, inv, "null arguments", name, None, cache(g), batch(g), *ws)
    refused(g, inv, "multiple", name, attn(q_heads=5, ld_q=320, ld_out=320), cache(g, heads=2, page_stride=2048), batch(g), *ws)
    refused(g, un, "64 or 128", name, attn(), cache(g, head_dim=32), batch(g), *ws)
    refused(g, un, "128 query heads", name, attn(q_heads=129, ld_q=1 << 20, ld_out=1 << 20), cache(g), batch(g), *ws)
    refused(g, un, "sequences", name, attn(), cache(g), batch(g, seqs=16385), *ws)
    refused(g, un, "2^40", name, attn(ld_q=1 << 41), cache(g), batch(g), *ws)
    for kw in (dict(q=A + 8), dict(out=B + 2), dict(ld_q=260), dict(hs_out=68, ld_out=512)):
        refused(g, al, "16-byte", name, attn(**kw), cache(g), batch(g), *ws)
    refused(g, al, "lse", name, attn(lse=S + 2), cache(g), batch(g), *ws)
    refused(g, al, "workspace", name, attn(), cache(g), batch(g), S + 8, 1 << 40)
    refused(g, inv, "negative workspace", name, attn(), cache(g), batch(g), S, -1)
    assert g.fp8_paged_attention(attn(), cache(g), batch(g, tokens=0), None, 0) == 0 and g.fp8_paged_attention(attn(), cache(g), batch(g, seqs=0), None, 0) == 0
    with pytest.raises(g.Fp8Error):
        g.fp8_paged_attention_workspace_bytes(attn(window=-1), cache(g), batch(g))


def test_attention_out_of_reach(g):
    def attn(**kw):
        return g.paged_attention(kw.pop("q_heads", 4), 0.125, **{**dict(q=A, ld_q=256, hs_q=64, out=B, ld_out=256, hs_out=64), **kw})
    name, ws, un = "fp8_paged_attention", (S, 1 << 50), g.FP8_ERR_UNSUPPORTED
    odd = dict(heads=2, head_stride=1024, pages=32768, page_stride=8 * 131101)  # a common part of 8: 2^32 of them
    refused(g, un, "common part", name, attn(), cache(g, **odd), batch(g), *ws)
    for kw in (dict(page_stride=1 << 39), dict(token_stride=1 << 35, page_stride=1 << 40)):
        refused(g, un, "2^39", name, attn(), cache(g, pages=2, **kw), batch(g), *ws)
    refused(g, un, "2^39", name, attn(ld_q=1 << 39), cache(g), batch(g), *ws)
    refused(g, g.FP8_ERR_INVALID_ARG, "in place", name, attn(out=A, ld_out=512), cache(g), batch(g), *ws)
    refused(g, un, "longer table", name, attn(), cache(g), batch(g, tokens=1 << 30, table_width=1 << 30, ld_table=1 << 30), *ws)
    a, c, b = attn(ld_q=1 << 39, hs_q=1 << 39, q_heads=1), cache(g, pages=1, page_stride=1 << 39, head_stride=1 << 39), batch(g, tokens=1)  # (strides that nothing uses)
    assert g.lib.fp8_paged_attention_workspace_bytes(a, c, b) >= 0


def test_blocks_of_tensors(g):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    x = z(4, 6, 64)
    f = g.qk_rope(4, 4, 1, 64, 64, g.FP8_DT_BF16, q=x[:, :4], k=x[:, 4:5], q_out=z(4, 4, 64).transpose(0, 1).contiguous().transpose(0, 1))
    assert (f.ld_q, f.hs_q, f.ld_k, f.hs_k, f.ld_q_out, f.hs_q_out) == (384, 64, 384, 64, 64, 256) and f.k == x.data_ptr() + 512
    for bad in (z(4, 3, 64), z(3, 4, 64), z(4, 4, 63), z(4, 256), z(4, 4, 128)[..., ::2]):
        with pytest.raises(ValueError):
            g.qk_rope(4, 4, 1, 64, 64, g.FP8_DT_BF16, q=bad)
    for kw in (dict(q=z(4, 4, 64, dt=torch.float16)), dict(pos=torch.zeros(4, dtype=torch.int64)), dict(turns=torch.zeros(32)), dict(w_q=z(64))):
        with pytest.raises(TypeError):
            g.qk_rope(4, 4, 1, 64, 64, g.FP8_DT_BF16, norm=1, **kw)
    for kw in (dict(pos=torch.zeros(3, dtype=torch.int32)), dict(turns=torch.zeros(31, dtype=torch.int64)), dict(w_q=torch.zeros(63))):
        with pytest.raises(ValueError):
            g.qk_rope(4, 4, 1, 64, 64, g.FP8_DT_BF16, norm=1, **kw)
    with pytest.raises(TypeError):
        g.qk_rope(4, 4, 1, 64, 64, g.FP8_DT_BF16, nothing=1)
    with pytest.raises(TypeError):
        g.qk_rope(4, 4, 1, 64, 64, g.FP8_DT_BF16, q=x, ld_q=384)
    c = g.kv_cache(z(9, 16, 2, 64).transpose(1, 2), z(9, 16, 2, 64).transpose(1, 2))
    assert (c.pages, c.heads, c.page_size, c.head_dim, c.page_stride, c.head_stride, c.token_stride, c.format) == (9, 2, 16, 64, 2048, 64, 128, 0)
    u8 = torch.uint8
    c = g.kv_cache(z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 2, dt=u8), z(9, 2, 16, 2, dt=u8))
    assert c.format == g.FP8_KV_MX_E4M3
    for args in ((z(9, 2, 16, 64), z(9, 2, 16, 128)), (z(9, 2, 16), z(9, 2, 16)), (z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 2, dt=u8)),
                 (z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 4, dt=u8), z(9, 2, 16, 4, dt=u8))):
        with pytest.raises(ValueError):
            g.kv_cache(*args)
    with pytest.raises(TypeError):
        g.kv_cache(z(9, 2, 16, 64, dt=u8), z(9, 2, 16, 64, dt=u8))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = g.kv_batch(7, i32(3), i32(2), i32(2, 9)[:, :5])
    assert (b.tokens, b.seqs, b.table_width, b.ld_table) == (7, 2, 5, 9)
    for args in ((7, i32(2), i32(2), i32(2, 5)), (7, i32(3), i32(2), i32(3, 5)), (7, i32(3), i32(2), i32(10))):
        with pytest.raises(ValueError):
            g.kv_batch(*args)
    with pytest.raises(TypeError):
        g.kv_batch(7, i32(3), i32(2).long(), i32(2, 5))
    a = g.paged_attention(4, 1.0, q=z(7, 4, 64), out=z(7, 4, 64), lse=torch.zeros(7, 4))
    cc = g.kv_cache(z(9, 2, 16, 64), z(9, 2, 16, 64))
    assert g.fp8_paged_attention_workspace_bytes(a, cc, b) >= 0
    for kw in (dict(q=z(6, 4, 64)), dict(out=z(7, 4, 32)), dict(lse=torch.zeros(6, 4))):
        with pytest.raises(ValueError):
            g.fp8_paged_attention_workspace_bytes(g.paged_attention(4, 1.0, **{**dict(q=z(7, 4, 64), out=z(7, 4, 64)), **kw}), cc, b)


def test_blocks_exchanged(g):
    f, c, b, a = g.qk_rope(0, 1, 1, 64, 0, 0), g.fp8_kv_cache_t(), g.fp8_kv_batch_t(), g.paged_attention(1, 1.0)
    grad = g.qk_rope_grad()
    for name, calls in (("fp8_kv_append", ((f, b, c), (c, c, b), (f, c, f), (bytes(512), c, b))), ("fp8_paged_attention", ((a, b, c, None, 0), (f, c, b, None, 0), (a, c, a, None, 0))),
                        ("fp8_qk_rope_fwd", ((grad,), (c,))), ("fp8_qk_rope_bwd", ((grad, f, None, 0), (f, f, None, 0)))):
        for fn in {getattr(g, name), getattr(g, "_by_ctypes", {}).get(name, getattr(g, name))}:
            for args in calls:
                with pytest.raises((TypeError, ctypes.ArgumentError)):
                    fn(*args)
