"""The operators between a block's projections as they are measured: what each case is, its inputs, its plain form in
elementary torch operations, the calls a user makes, and the same results in 64 bits.

Operators (one dict per case, "op" says which):
  rope       queries and keys as the QKV projection writes them: the norm over each head (root mean square with a weight, or none) and
             the rotation by the token's position, in one pass; "bwd": the gradients of the same.
  append     the same on the way into a paged cache: queries out, keys (normed, rotated) and values into the slots of the new tokens.
  attend     attention of the new tokens of each sequence (one token each, or a chunk) over its paged cache, causal at the
             cache's end, optionally within a window.
  step       append, then attend, over a cache of 8-bit codes: one layer's attention while tokens are generated.

Conventions: token i of a sequence's n new ones sits at position len - n + i, len counting the new tokens. The cache is [pages, heads,
page, D] for keys and for values, in bf16 ("bf16") or as E4M3 codes with one power of two per 32 elements along D ("mx": the smallest 2^e
with 448 2^e >= the group's amax, stored as e + 127). Frequencies are base^(-2i/R); "parts" divides those that turn less
than `low` times over `orig` positions by `factor`, leaves those that turn more than `high` times, and goes between the two linearly.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
LOW, HIGH = 1.0, 4.0


def listed():
    return [
        # a training batch of four sequences through one layer, grouped heads, in place of the projection's output
        dict(name="rope training", op="rope", way="fwd", T=16384, Hq=32, Hk=8, D=128, R=128, layout="half", norm=True, dt="bf16", base=500000.0, factor=1.0, orig=0, start=0, seq=4096),
        # a ragged batch late in a long context: part of the head rotated in pairs, stretched frequencies, no norm, fp32
        dict(name="rope long context partial", op="rope", way="fwd", T=1021, Hq=12, Hk=12, D=64, R=32, layout="pairs", norm=False, dt="f32", base=10000.0, factor=8.0, orig=8192, start=1048576, seq=1021),
        # the training batch's backward, with the weights' gradients
        dict(name="rope backward training", op="rope", way="bwd", T=16384, Hq=32, Hk=8, D=128, R=128, layout="half", norm=True, dt="bf16", base=500000.0, factor=1.0, orig=0, start=0, seq=4096),
        # the backward of a small model's batch: 12 heads of 64, rotated in pairs, odd number of tokens
        dict(name="rope backward small", op="rope", way="bwd", T=4099, Hq=12, Hk=12, D=64, R=64, layout="pairs", norm=True, dt="f32", base=10000.0, factor=1.0, orig=0, start=0, seq=1024),
        # a long prompt's chunk into an empty bf16 cache
        dict(name="append prompt", op="append", B=1, q=8192, ragged=False, old=0, Hq=32, Hk=8, D=128, R=128, layout="half", norm=True, page=64, base=500000.0, factor=1.0, orig=0),
        # one new token for each of 64 running sequences
        dict(name="append one token each", op="append", B=64, q=1, ragged=True, old=4095, Hq=32, Hk=8, D=128, R=128, layout="half", norm=True, page=16, base=500000.0, factor=8.0, orig=8192),
        # one sequence, one token, a short past: the latency of a single user's step
        dict(name="attend one token", op="attend", B=1, q=1, ragged=False, old=1000, Hq=32, Hk=8, D=128, cache="bf16", page=16, window=0),
        # the tokens of 64 running sequences of very different lengths
        dict(name="attend batch of tokens", op="attend", B=64, q=1, ragged=True, old=8191, Hq=32, Hk=8, D=128, cache="bf16", page=64, window=0),
        # a chunk of a long prompt over what came before it
        dict(name="attend chunk", op="attend", B=1, q=2048, ragged=False, old=14336, Hq=32, Hk=8, D=128, cache="bf16", page=128, window=0),
        # first chunks and single tokens in one batch, small heads in odd groups, a window, 8-bit cache
        dict(name="attend mixed in a window", op="attend", B=24, q=700, ragged=True, old=3000, Hq=15, Hk=5, D=64, cache="mx", page=32, window=1500),
        # one step of a large batch over an 8-bit cache
        dict(name="step of a batch", op="step", B=96, q=1, ragged=True, old=8191, Hq=32, Hk=8, D=128, R=128, layout="half", norm=True, cache="mx", page=64, window=0, base=500000.0, factor=8.0, orig=8192),
        # one user's step far into a long context: few rows over a long axis
        dict(name="step one long context", op="step", B=1, q=1, ragged=False, old=131071, Hq=32, Hk=8, D=128, R=128, layout="half", norm=True, cache="mx", page=64, window=0, base=500000.0, factor=8.0, orig=8192),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "attend", "attend", "attend", "step"])
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 5, 8, 12])
    Hq = Hk * rng.choice([1, 2, 3, 4, 7, 8])
    long = rng.random() < 0.5
    turn = dict(R=D if rng.random() < 0.7 else D // 2, layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6, base=rng.choice([10000.0, 500000.0]),
                factor=8.0 if long else 1.0, orig=8192 if long else 0)
    if op == "rope":
        T = _log(rng, 1, 16384)
        while T * (Hq + Hk) * D > 16384 * 40 * 128:
            T = max(1, T // 2)
        return dict(op=op, way=rng.choice(["fwd", "bwd"]), T=T, Hq=Hq, Hk=Hk, D=D, dt=rng.choice(["bf16", "bf16", "f32"]), start=rng.choice([0, _log(rng, 1, 1 << 20)]),
                    seq=_log(rng, 1, T), **turn)
    B = _log(rng, 1, 128)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        q = rng.choice([1, _log(rng, 1, 8192)])
        case = dict(op=op, B=B, q=q, ragged=rng.random() < 0.7, old=rng.choice([0, _log(rng, 1, 4096)]), Hq=Hq, Hk=Hk, D=D, page=page, **turn)
        while case["B"] * case["q"] * (Hq + 2 * Hk) * D > 8192 * 48 * 128 or case["B"] * (case["q"] + case["old"]) * Hk * D > 64 * 4096 * 1024:
            case["B"], case["old"] = max(1, case["B"] // 2), case["old"] // 2
            case["q"] = max(1, case["q"] * 3 // 4)
        return case
    q = 1 if op == "step" else rng.choice([1, rng.randint(2, 8), _log(rng, 8, 2048)])
    case = dict(op=op, B=B, q=q, ragged=rng.random() < 0.7, old=_log(rng, 1, 65536), Hq=Hq, Hk=Hk, D=D, cache="mx" if op == "step" else rng.choice(["bf16", "mx"]), page=page,
                window=rng.choice([0, 0, _log(rng, 1, 8192)]))
    if op == "step":
        case.update(turn)
    for _ in range(40):
        rows, length = case["B"] * case["q"], case["old"] + case["q"]
        if rows * Hq * length <= 2048 * 32 * 15000 and case["B"] * length * Hk * D <= 64 * 8192 * 1024:
            break
        case["B"], case["old"], case["q"] = max(1, case["B"] * 3 // 4), max(1, case["old"] * 3 // 4), max(1, case["q"] * 7 // 8)
    return case


# ------------------------------------------------------------------------------------------------
# a batch's lengths
# ------------------------------------------------------------------------------------------------
def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence. Ragged: spread between an eighth and the whole,
    every fourth sequence with a single new token."""
    B, q, old = case["B"], case["q"], case["old"]
    if not case["ragged"]:
        return [q] * B, [old + q] * B
    part = [((i + 1) * 0.6180339887 % 1.0) for i in range(B)]
    new = [1 if i % 4 == 3 else max(1, round(q * (0.125 + 0.875 * p))) for i, p in enumerate(part)]
    past = [round(old * (0.125 + 0.875 * ((p * 7.31) % 1.0))) for p in part]
    return new, [a + b for a, b in zip(new, past)]


def _allowed(new, total, window):
    """Pairs of a query and a key that it attends to, over all sequences."""
    n = 0
    for a, t in zip(new, total):
        for first, last in ((t - a + 1, t),):  # keys of the first and of the last query, without a window
            if window and window < last:
                short = max(0, min(window, last) - first + 1) if first <= window else 0
                n += sum((first, first + short - 1)) * short // 2 + (a - short) * window
            else:
                n += (first + last) * a // 2
    return n


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _frequencies(case):
    """Radians a position, [R / 2] in 64 bits."""
    i = torch.arange(case["R"] // 2, dtype=torch.float64, device="cuda")
    f = case["base"] ** (-2.0 * i / case["R"])
    if case["factor"] != 1.0:
        keep = ((case["orig"] * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / case["factor"])
    return f


def _turn_inputs(s, gen, T, dt):
    """A projection's output rows [T, Hq + 2 Hk heads], its parts, and what turns them."""
    Hq, Hk, D = s["Hq"], s["Hk"], s["D"]
    size = torch.exp(0.4 * _normal(gen, (Hq + 2 * Hk) * D))
    s["x"] = (_normal(gen, T, (Hq + 2 * Hk) * D) * size).to(dt).view(T, Hq + 2 * Hk, D)
    s["q"], s["k"], s["v"] = s["x"][:, :Hq], s["x"][:, Hq : Hq + Hk], s["x"][:, Hq + Hk :]
    s["w_q"], s["w_k"] = (1 + 0.2 * _normal(gen, D), 1 + 0.2 * _normal(gen, D)) if s["norm"] else (None, None)
    s["freq"] = _frequencies(s)
    s["amplitude"] = 1.0 + 0.1 * math.log(s["factor"]) if s["factor"] > 1 else 1.0


def _to_mx(x):
    """x [..., D] fp32 -> E4M3 elements (the numbers, before their scale) and e per 32 of them."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    m, e = torch.frexp(g.abs().amax(dim=-1))  # a = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    e = torch.where(m == 0, torch.zeros_like(e), e)
    return torch.ldexp(g, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), e


def _from_mx(codes, e):
    """[..., D / 32, 32] elements and their e -> fp32 values [..., D]."""
    return torch.ldexp(codes.float(), e.unsqueeze(-1)).flatten(-2)


def _cache_inputs(s, gen):
    """Pages of recycled memory with what the sequences hold, their table, and the batch's lengths on the device."""
    new, total = _lengths(s)
    P, Hk, D = s["page"], s["Hk"], s["D"]
    need = [-(-n // P) for n in total]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    first = torch.tensor([sum(need[:i]) for i in range(s["B"])], device="cuda").unsqueeze(1)
    col = torch.arange(width, device="cuda").unsqueeze(0)
    held = col < torch.tensor(need, device="cuda").unsqueeze(1)
    s["table"] = torch.where(held, order[torch.where(held, first + col, torch.zeros_like(col))], torch.full_like(order[:1], -1))
    s["start"] = torch.tensor([sum(new[:i]) for i in range(s["B"] + 1)], dtype=torch.int32, device="cuda")
    s["len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["T"], s["qmax"], s["lmax"] = sum(new), max(new), max(total)
    for n in ("kc", "vc"):
        x = _normal(gen, pages, Hk, P, D)
        if s.get("cache", "bf16") == "mx":
            codes, e = _to_mx(x * torch.exp(0.4 * _normal(gen, D)))
            s[n], s[n + "s"] = codes.view(torch.uint8).flatten(-2), (e + 127).to(torch.uint8)
        else:
            s[n] = x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    new = lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    if case["op"] == "rope":
        T, Hq, Hk, D, dt = case["T"], case["Hq"], case["Hk"], case["D"], DT[case["dt"]]
        _turn_inputs(s, gen, T, dt)
        s["pos"] = (case["start"] + torch.arange(T, device="cuda") % case["seq"]).to(torch.int32)
        s["y"] = new(T, Hq + Hk, D, dt=dt)
        s["q_out"], s["k_out"] = s["y"][:, :Hq], s["y"][:, Hq:]
        if case["way"] == "bwd":
            s["dy"] = (0.01 * _normal(gen, T, Hq + Hk, D)).to(dt)
            s["dx"] = new(T, Hq + Hk, D, dt=dt)
            s["dw_q"], s["dw_k"] = (new(D), new(D)) if case["norm"] else (None, None)
    else:
        _cache_inputs(s, gen)
        T, Hq, D = s["T"], case["Hq"], case["D"]
        if case["op"] == "attend":
            s["q_out"] = (1.5 * _normal(gen, T, Hq, D)).to(torch.bfloat16)
        else:
            _turn_inputs(s, gen, T, torch.bfloat16)
            s["q_out"] = new(T, Hq, D, dt=torch.bfloat16)
        if case["op"] != "append":
            s["out"], s["lse"] = new(T, Hq, D, dt=torch.bfloat16), new(T, Hq)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The argument blocks that a user's program keeps for a layer."""
    import fp8_mixed_precision_saturating_gb300 as g
    if s["op"] != "attend":
        kind = g.FP8_ROPE_PARTS if s["factor"] != 1.0 else g.FP8_ROPE_PLAIN
        turns = g.rope_turns(s["R"], s["base"], kind, s["factor"], s["orig"], LOW, HIGH, device="cuda")
        more = dict(k_out=s["k_out"], pos=s["pos"]) if s["op"] == "rope" else dict(v=s["v"])
        s["plan"] = g.qk_rope(
            s["T"], s["Hq"], s["Hk"], s["D"], s["R"], g.FP8_DT_F32 if s.get("dt") == "f32" else g.FP8_DT_BF16,
            layout=g.FP8_ROPE_INTERLEAVED if s["layout"] == "pairs" else g.FP8_ROPE_HALF, norm=g.FP8_NORM_RMS if s["norm"] else g.FP8_NORM_NONE, eps=EPS,
            amplitude=s["amplitude"], turns=turns, q=s["q"], k=s["k"], w_q=s["w_q"], w_k=s["w_k"], q_out=s["q_out"], **more)
    if s["op"] == "rope":
        if s["way"] == "bwd":
            Hq = s["Hq"]
            s["back"] = g.qk_rope_grad(dq_out=s["dy"][:, :Hq], dk_out=s["dy"][:, Hq:], dq=s["dx"][:, :Hq], dk=s["dx"][:, Hq:], dw_q=s["dw_q"], dw_k=s["dw_k"])
            s["ws"] = torch.empty(max(16, g.fp8_qk_rope_bwd_workspace_bytes(s["plan"], s["back"])), dtype=torch.uint8, device="cuda")
        return
    s["cache_plan"] = g.kv_cache(s["kc"], s["vc"], s.get("kcs"), s.get("vcs"))
    s["batch_plan"] = g.kv_batch(s["T"], s["start"], s["len"], s["table"])
    if s["op"] != "append":
        s["attend_plan"] = g.paged_attention(s["Hq"], 1.0 / math.sqrt(s["D"]), window=s["window"], q=s["q_out"], out=s["out"], lse=s["lse"])
        n = g.fp8_paged_attention_workspace_bytes(s["attend_plan"], s["cache_plan"], s["batch_plan"])
        s["ws"] = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _angles(s, pos):
    """cos and sin [T, 1, R / 2] in fp32; the angles of far positions need 64 bits."""
    a = pos.double().unsqueeze(1) * s["freq"]
    return (torch.cos(a) * s["amplitude"]).float().unsqueeze(1), (torch.sin(a) * s["amplitude"]).float().unsqueeze(1)


def _halves(s, x):
    """The two members of each rotated pair, and the rest of the head."""
    R = s["R"]
    if s["layout"] == "half":
        return x[..., : R // 2], x[..., R // 2 : R], x[..., R:]
    return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]


def _joined(s, a, b, rest):
    both = torch.cat([a, b], dim=-1) if s["layout"] == "half" else torch.stack([a, b], dim=-1).flatten(-2)
    return torch.cat([both, rest], dim=-1)


def _turned(s, x, cos, sin):
    a, b, rest = _halves(s, x)
    return _joined(s, a * cos - b * sin, a * sin + b * cos, rest)


def _root(x):
    return 1.0 / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / x.shape[-1] + EPS)


def _normed(s, x, w):
    return x * _root(x) * w if s["norm"] else x


def _plain_rope(s):
    cos, sin = _angles(s, s["pos"])
    q, k = s["q"].float(), s["k"].float()
    if s["way"] == "fwd":
        return {n: _turned(s, _normed(s, x, s["w_" + n]), cos, sin).to(DT[s["dt"]]) for n, x in (("q", q), ("k", k))}
    out = {}
    for n, x, dy in (("q", q, s["dy"][:, : s["Hq"]].float()), ("k", k, s["dy"][:, s["Hq"] :].float())):
        dn = _turned(s, dy, cos, -sin)
        if s["norm"]:
            r = _root(x)
            z = x * r
            out["dw_" + n] = (dn * z).sum(dim=(0, 1))
            dz = dn * s["w_" + n]
            dn = r * (dz - z * ((dz * z).sum(dim=-1, keepdim=True) / x.shape[-1]))
        out["d" + n] = dn.to(DT[s["dt"]])
    return out


def _places(s):
    """For each new token its sequence and its position in it."""
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(s["start"][1:].contiguous(), t.int(), right=True)
    return seq, s["len"].long()[seq] - s["start"].long()[seq + 1] + t


def _new_rows(s):
    seq, pos = _places(s)
    cos, sin = _angles(s, pos)
    q = _turned(s, _normed(s, s["q"].float(), s["w_q"]), cos, sin).to(torch.bfloat16)
    k = _turned(s, _normed(s, s["k"].float(), s["w_k"]), cos, sin)
    return q, k, s["v"].float(), s["table"].long()[seq, pos // s["page"]], pos % s["page"]


def _plain_append(s):
    q, k, v, page, slot = _new_rows(s)
    s["kc"][page, :, slot] = k.to(torch.bfloat16)
    s["vc"][page, :, slot] = v.to(torch.bfloat16)
    return {"q": q, "k": s["kc"], "v": s["vc"]}


def _values(s, name, page, slot):
    """What the cache holds at the places given, in fp32."""
    x = s[name][page, :, slot]
    if s["cache"] == "bf16":
        return x.float()
    return _from_mx(x.view(torch.float8_e4m3fn).unflatten(-1, (-1, 32)), s[name + "s"][page, :, slot].int() - 127)


def _plain_attend(s):
    B, P, Hq, Hk, D, Q, L = s["B"], s["page"], s["Hq"], s["Hk"], s["D"], s["qmax"], s["lmax"]
    G = Hq // Hk
    key = torch.arange(L, device="cuda")
    page = s["table"].long()[:, key // P].clamp(min=0)
    k, v = (_values(s, n, page, (key % P).expand(B, L)).transpose(1, 2) for n in ("kc", "vc"))  # [B, Hk, L, D]
    new, total = (s["start"][1:] - s["start"][:-1]).long(), s["len"].long()
    row = torch.arange(Q, device="cuda").unsqueeze(0)
    at = (s["start"][:-1].long().unsqueeze(1) + row).clamp(max=s["T"] - 1)
    q = s["q_out"].float()[at].view(B, Q, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, Q * G, D)
    pos = (total - new).unsqueeze(1) + row
    sees = (key <= pos.unsqueeze(2)) & (row < new.unsqueeze(1)).unsqueeze(2)
    if s["window"]:
        sees &= key > pos.unsqueeze(2) - s["window"]
    w = torch.matmul(q, k.transpose(2, 3)).view(B, Hk, Q, G, L) * (1.0 / math.sqrt(D))
    w = w.masked_fill(~sees.view(B, 1, Q, 1, L), -math.inf)
    top = w.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    w = torch.exp(w - top)
    total_w = w.sum(dim=-1, keepdim=True)
    v = v.masked_fill((key >= total.unsqueeze(1)).view(B, 1, L, 1), 0.0)
    o = torch.matmul(w.view(B, Hk, Q * G, L), v).view(B, Hk, Q, G, D) / total_w.clamp(min=torch.finfo(torch.float32).tiny)
    lse = (torch.log(total_w) + top).squeeze(-1)
    here = torch.nonzero((row < new.unsqueeze(1)).view(-1)).squeeze(1)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * Q, Hq, D)[here]
    return {"out": o.to(torch.bfloat16), "lse": lse.permute(0, 2, 1, 3).reshape(B * Q, Hq)[here]}


def _plain_step(s):
    q, k, v, page, slot = _new_rows(s)
    s["q_out"].copy_(q)
    for n, x in (("kc", k), ("vc", v)):
        codes, e = _to_mx(x)
        s[n][page, :, slot] = codes.view(torch.uint8).flatten(-2)
        s[n + "s"][page, :, slot] = (e + 127).to(torch.uint8)
    return {"q": s["q_out"], **_plain_attend(s)}


def _own_rope(s):
    import fp8_mixed_precision_saturating_gb300 as g
    if s["way"] == "fwd":
        g.fp8_qk_rope_fwd(s["plan"])
        return {"q": s["q_out"], "k": s["k_out"]}
    g.fp8_qk_rope_bwd(s["plan"], s["back"], s["ws"], s["ws"].numel())
    out = {"dq": s["dx"][:, : s["Hq"]], "dk": s["dx"][:, s["Hq"] :]}
    if s["norm"]:
        out.update(dw_q=s["dw_q"], dw_k=s["dw_k"])
    return out


def _own_append(s):
    import fp8_mixed_precision_saturating_gb300 as g
    g.fp8_kv_append(s["plan"], s["cache_plan"], s["batch_plan"])
    return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}


def _own_attend(s):
    import fp8_mixed_precision_saturating_gb300 as g
    g.fp8_paged_attention(s["attend_plan"], s["cache_plan"], s["batch_plan"], s["ws"], s["ws"].numel())
    return {"out": s["out"], "lse": s["lse"]}


def _own_step(s):
    import fp8_mixed_precision_saturating_gb300 as g
    g.fp8_kv_append(s["plan"], s["cache_plan"], s["batch_plan"])
    return {"q": s["q_out"], **_own_attend(s)}


_plain = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "step": _plain_step}
_own = {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "step": _own_step}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "rope":
        size, n = {"bf16": 2, "f32": 4}[case["dt"]], case["T"] * (Hq + Hk) * D
        # forward: in and out; backward: the gradient in and out, and with a norm its input
        return {"bytes": n * size * (3 if case["way"] == "bwd" and case["norm"] else 2) + 4 * case["T"] + 4 * case["R"], "flops": n * (20 if case["way"] == "bwd" else 10)}
    new, total = _lengths(case)
    T, elem = sum(new), 1 + 1 / 32 if case.get("cache") == "mx" else 2
    bytes_, flops = 0, 0
    if case["op"] != "attend":
        bytes_ += T * (2 * Hq + 2 * Hk) * D * 2 + 2 * T * Hk * D * elem
        flops += 10 * T * (Hq + 2 * Hk) * D
    if case["op"] != "append":
        w = case["window"]
        read = sum(min(t, w + a - 1) if w else t for a, t in zip(new, total))
        bytes_ += 2 * read * Hk * D * elem + T * Hq * (4 * D + 4) + 4 * sum(-(-t // case["page"]) for t in total)
        flops += 4 * D * Hq * _allowed(new, total, w)
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------------------------
# in 64 bits, from the definitions
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    return _exact(case, prepare(case, seed))


def _rotation64(case, pos):
    """The rotations as complex numbers [T, 1, R / 2]."""
    R = case["R"]
    f = torch.tensor([case["base"] ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64, device="cuda")
    if case["factor"] != 1.0:
        turns = case["orig"] * f / (2 * math.pi)
        share = torch.where(turns < LOW, torch.zeros_like(f), torch.where(turns > HIGH, torch.ones_like(f), (turns - LOW) / (HIGH - LOW)))
        f = share * f + (1 - share) * (f / case["factor"])
    size = 1.0 + 0.1 * math.log(case["factor"]) if case["factor"] > 1 else 1.0
    return torch.polar(torch.full((pos.numel(), R // 2), size, dtype=torch.float64, device="cuda"), torch.outer(pos.double(), f)).unsqueeze(1)


def _rows64(case, x, w, z):
    """Norm and rotation of heads [T, H, D]; z: the rotations."""
    if case["norm"]:
        x = w * (x / (x.pow(2).mean(dim=-1, keepdim=True) + EPS).sqrt())
    R, T, H = case["R"], x.shape[0], x.shape[1]
    first = x[..., :R]
    pairs = first.reshape(T, H, 2, R // 2).transpose(2, 3) if case["layout"] == "half" else first.reshape(T, H, R // 2, 2)
    c = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    c = c.transpose(2, 3) if case["layout"] == "half" else c
    return torch.cat([c.reshape(T, H, R), x[..., R:]], dim=-1)


def _rounded64(x):
    """The values of the 8-bit form: for each 32 along the last axis, multiples of a power of two with three bits after the leading one."""
    g = x.reshape(-1, 32)
    top = g.abs().max(dim=1, keepdim=True).values
    unit = torch.exp2(torch.ceil(torch.log2(top / 448)))
    unit = torch.where(448 * unit < top, 2 * unit, torch.where(448 * (unit / 2) >= top, unit / 2, unit))
    y = g / unit
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(top > 0, torch.round(y / step) * step * unit, torch.zeros_like(g)).reshape(x.shape)


def _decoded64(s, name, page, slot):
    x = s[name][page, :, slot]
    if s["cache"] == "bf16":
        return x.double()
    b = x.int()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(8 + m, e - 10))
    scale = torch.exp2(s[name + "s"][page, :, slot].double() - 127)
    return torch.where(b >= 128, -mag, mag) * scale.repeat_interleave(32, dim=-1)


def _exact(case, s):
    if case["op"] == "rope":
        z = _rotation64(case, s["pos"])
        if case["way"] == "fwd":
            return {n: _rows64(case, s[n].double(), None if s["w_" + n] is None else s["w_" + n].double(), z) for n in ("q", "k")}
        out = {}
        with torch.enable_grad():
            for n, dy in (("q", s["dy"][:, : case["Hq"]]), ("k", s["dy"][:, case["Hq"] :])):
                x = s[n].double().requires_grad_(True)
                w = s["w_" + n].double().requires_grad_(True) if case["norm"] else None
                d = torch.autograd.grad(_rows64(case, x, w, z), [x] + ([w] if case["norm"] else []), dy.double())
                out["d" + n] = d[0]
                if case["norm"]:
                    out["dw_" + n] = d[1]
        return out
    new, total = _lengths(case)
    P = case["page"]
    out, new_k, new_v = {}, {}, {}
    if case["op"] != "attend":
        pos = torch.cat([torch.arange(t - a, t, device="cuda") for a, t in zip(new, total)])
        z = _rotation64(case, pos)
        out["q"] = _rows64(case, s["q"].double(), None if s["w_q"] is None else s["w_q"].double(), z)
        k, v = _rows64(case, s["k"].double(), None if s["w_k"] is None else s["w_k"].double(), z), s["v"].double()
        seq = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), torch.tensor(new, device="cuda"))
        page, slot = s["table"].long()[seq, pos // P], pos % P
        if case["op"] == "append":
            out["k"], out["v"] = s["kc"].double(), s["vc"].double()
            out["k"][page, :, slot] = k
            out["v"][page, :, slot] = v
            return out
        new_k, new_v = (dict(enumerate(torch.split(_rounded64(x), new))) for x in (k, v))
        s["q_out"].copy_(out["q"])  # the attention reads the stored queries
    rows, lses = [], []
    first, G = 0, case["Hq"] // case["Hk"]
    for b, (a, t) in enumerate(zip(new, total)):
        key = torch.arange(t, device="cuda")
        page = s["table"].long()[b, key // P]
        k, v = _decoded64(s, "kc", page, key % P), _decoded64(s, "vc", page, key % P)
        if case["op"] == "step":
            k[t - a :], v[t - a :] = new_k[b], new_v[b]
        at = torch.arange(t - a, t, device="cuda").unsqueeze(1)
        hidden = (key > at) | ((key <= at - case["window"]) if case["window"] else torch.zeros_like(key > at))
        o, l = [], []
        for h in range(case["Hq"]):
            w = (s["q_out"][first : first + a, h].double() @ k[:, h // G].T) / math.sqrt(case["D"])
            w[hidden] = -math.inf
            l.append(torch.logsumexp(w, dim=1))
            o.append(torch.softmax(w, dim=1) @ v[:, h // G])
        rows.append(torch.stack(o, dim=1))
        lses.append(torch.stack(l, dim=1))
        first += a
    out.update(out=torch.cat(rows), lse=torch.cat(lses))
    return out
