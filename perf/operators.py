"""The 4-bit and block-norm operators as they are measured: what each case is, its inputs, its plain
form in elementary torch operations, the calls a user makes, and the same results in 64 bits.

Operators (one dict per case, "op" says which):
  quantize   bf16 -> microscaled 4-bit codes and back to the values they stand for. NVFP4 ("nv"): E2M1
             codes, one E4M3 scale per 16 elements, optionally one fp32 scale for the tensor. MXFP4
             ("mx"): E2M1 codes, one power of two per 32. Groups run along the rows (an activation, whose
             contraction is its columns), down the columns (a weight [K, N], codes written transposed)
             or both (a gradient, which the backward contracts both ways).
  mm         C = A B^T of two such operands along their common contraction.
  norm_fwd   n = norm(o), r' = alpha r + gate n, h = norm(r'): what stands between one block's
             output o and the next block's input h on the residual stream r; with "emit", h goes straight
             into 4 bits and through the next projection.
  norm_bwd   its gradients.

Row-major everywhere. 4-bit operands: element k of a row is the low (k even) or high nibble of byte k / 2, rows
padded with zero codes to 16 bytes (32 elements); scale bytes in atoms of 512: atom (row / 128, g / 4), g the group's
index along the contraction, holds the byte of (row, g) at 16 (row % 32) + 4 ((row / 32) % 4) + g % 4.
"""
import math

import torch

own = False

GROUP = {"nv": 16, "mx": 32}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # activations of one training batch into 4 bits, and back (a saved activation read by the backward)
        dict(name="quantize activations", op="quantize", fmt="nv", rows=16384, cols=4096, along="rows", scaling="none"),
        # a weight cache refresh after an optimizer step: one scale from the whole tensor, groups along K
        dict(name="quantize weight", op="quantize", fmt="nv", rows=4096, cols=14336, along="cols", scaling="current"),
        # a gradient that dgrad contracts along its rows and wgrad down its columns, ragged batch
        dict(name="quantize gradient ragged", op="quantize", fmt="mx", rows=4099, cols=1536, along="both", scaling="none"),
        # one new token through an up-projection: the weights' bytes and the latency count
        dict(name="product one token", op="mm", fmt="nv", M=1, N=14336, K=4096, out="bf16", scaled=True),
        # a small batch of tokens being generated
        dict(name="product few tokens", op="mm", fmt="mx", M=23, N=6144, K=1536, out="bf16", scaled=False),
        # the forward of a training batch at full size
        dict(name="product training forward", op="mm", fmt="nv", M=16384, N=14336, K=4096, out="bf16", scaled=True),
        # a weight gradient: few outputs, a long ragged contraction over the tokens, fp32 result
        dict(name="product weight gradient", op="mm", fmt="nv", M=1536, N=1000, K=16379, out="f32", scaled=True),
        # one token between two blocks, into the next block's 4-bit up-projection
        dict(name="norm one token into 4 bits", op="norm_fwd", T=1, D=4096, post="rms", pre="rms", stream="bf16", block="bf16",
             gate_rows=1 << 30, alpha=True, emit="nv", N=4096),
        # a training batch between two blocks
        dict(name="norm training", op="norm_fwd", T=16384, D=4096, post="rms", pre="rms", stream="bf16", block="bf16",
             gate_rows=1 << 30, alpha=True, emit="", N=0),
        # a GPT-2-like stream kept in fp32, layer norms, a gate for each sequence, odd width
        dict(name="norm odd fp32 stream", op="norm_fwd", T=4099, D=1537, post="none", pre="layer", stream="f32", block="bf16",
             gate_rows=1024, alpha=False, emit="", N=0),
        # the training batch's backward
        dict(name="norm backward training", op="norm_bwd", T=16384, D=4096, post="rms", pre="rms", stream="bf16", block="bf16",
             gate_rows=1 << 30, alpha=True),
        # the backward of sequences of uneven number with their own gates, layer norms, fp32 stream
        dict(name="norm backward sequences", op="norm_bwd", T=4100, D=1536, post="layer", pre="layer", stream="f32", block="bf16",
             gate_rows=500, alpha=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "mm", "norm_fwd", "norm_bwd"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 16384), _log(rng, 32, 14336)
        if rng.random() < 0.5:  # as often aligned as not
            cols = -(-cols // 32) * 32
        while rows * cols > 16384 * 4096:
            rows //= 2
        fmt = rng.choice(["nv", "mx"])
        return dict(op=op, fmt=fmt, rows=rows, cols=cols, along=rng.choice(["rows", "cols", "both"]),
                    scaling=rng.choice(["none", "current"]) if fmt == "nv" else "none")
    if op == "mm":
        M, N, K = _log(rng, 1, 16384), _log(rng, 16, 14336), _log(rng, 32, 16384)
        if rng.random() < 0.5:
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        while M * N * K > 16384 * 14336 * 4096:
            M //= 2
        return dict(op=op, fmt=rng.choice(["nv", "mx"]), M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]), scaled=rng.random() < 0.5)
    T, D = _log(rng, 1, 16384), _log(rng, 32, 8192)
    if rng.random() < 0.7:
        D = -(-D // 32) * 32
    while T * D > 16384 * 4096:
        T //= 2
    case = dict(op=op, T=T, D=D, post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]), stream=rng.choice(["bf16", "f32"]),
                block="bf16", gate_rows=rng.choice([0, 1 << 30, _log(rng, 1, 2048)]), alpha=rng.random() < 0.5)
    if case["stream"] == "f32" and rng.random() < 0.3:
        case["block"] = "f32"
    if op == "norm_fwd":
        emit = rng.choice(["", "nv", "mx"]) if D % 32 == 0 else ""
        case.update(emit=emit, N=_log(rng, 16, 4096) if emit else 0)
    return case


# ------------------------------------------------------------------------------------------------
# 4-bit numbers in elementary operations, fp32
# ------------------------------------------------------------------------------------------------
def _e2m1(v):
    """Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, saturating), with v's sign."""
    a = v.abs()
    m = 0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
    m += (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float()
    return torch.where(v < 0, -m, m)


def _pow2(e):
    """2^e in fp32 for whole e of -127 .. 127, by its bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantize(x, fmt, s):
    """x [R, C] fp32, groups along C -> element values [R, G, group] and scales [R, G], both as the numbers they stand for."""
    g = GROUP[fmt]
    R, C = x.shape
    G = -(-C // g)
    x = torch.nn.functional.pad(x, (0, G * g - C)).view(R, G, g)
    a = x.abs().amax(dim=2)
    if fmt == "nv":
        c = ((a * s) / torch.full_like(a, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        r = torch.where(c > 0, s / c, torch.zeros_like(c))
        return _e2m1(x * r.unsqueeze(2)), c
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1): the smallest power of two whose 6 times reaches a
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(min=-127)
    e = torch.where(a == 0, torch.zeros_like(e), e)
    return _e2m1(x * _pow2(-e).unsqueeze(2)), _pow2(e)


def _tensor_scale(x, scaling):
    one = torch.ones(1, device=x.device)
    if scaling == "none" or x.numel() == 0:
        return one, one
    a, top = x.abs().amax().float().view(1), torch.full((1,), 2688.0, device=x.device)
    return torch.where(a > 0, top / a, one), torch.where(a > 0, a / top, one)


_CODE = {0.0: 0, 0.5: 1, 1.0: 2, 1.5: 3, 2.0: 4, 3.0: 5, 4.0: 6, 6.0: 7}


def _pack(q, c, fmt, C):
    """Element values and scales as the bytes of a 4-bit operand: codes [R, row bytes] and scale atoms."""
    R, G, g = q.shape
    dev = q.device
    table = torch.zeros(13, dtype=torch.uint8, device=dev)
    for v, n in _CODE.items():
        table[int(2 * v)] = n
    codes = table[(q.abs() * 2).long()] | ((q < 0).to(torch.uint8) << 3)
    width = -(-C // 32) * 32
    codes = torch.nn.functional.pad(codes.view(R, G * g), (0, max(0, width - G * g)))[:, :width]
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    if fmt == "nv":
        byte, fill = c.to(torch.float8_e4m3fn).view(torch.uint8), 0
    else:
        byte, fill = (torch.frexp(c)[1] + 126).to(torch.uint8), 127
    nb, na = -(-R // 128), -(-G // 4)
    full = torch.full((nb * 128, na * 4), fill, dtype=torch.uint8, device=dev)
    full[:R, :G] = byte
    atoms = full.view(nb, 4, 32, na, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return packed.contiguous(), atoms


def _unpack(packed, atoms, fmt, R, C):
    """The values [R, C] in fp32 that the bytes of a 4-bit operand stand for (without a tensor scale)."""
    g = GROUP[fmt]
    G = -(-C // g)
    nb, na = -(-R // 128), -(-G // 4)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=packed.device)
    codes = torch.stack([packed & 15, packed >> 4], dim=2).view(R, -1)
    v = table[codes.int()][:, :C]
    b = atoms.view(nb, na, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(nb * 128, na * 4)[:R, :G]
    c = b.contiguous().view(torch.float8_e4m3fn).float() if fmt == "nv" else _pow2(b.int() - 127)
    return v * c.repeat_interleave(g, dim=1)[:, :C]


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _operand(gen, fmt, R, C, std):
    """A 4-bit operand of normal values whose columns have different sizes, as quantised before the call."""
    x = _normal(gen, R, C) * (std * torch.exp(0.5 * _normal(gen, C)))
    s, d = _tensor_scale(x, "current" if fmt == "nv" else "none")
    q, c = _quantize(x, fmt, s)
    return (*_pack(q, c, fmt, C), d)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    new = lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    u8 = lambda *shape: new(*shape, dt=torch.uint8)  # noqa: E731
    if case["op"] == "quantize":
        R, C, fmt = case["rows"], case["cols"], case["fmt"]
        s["x"] = (_normal(gen, R, C) * torch.exp(_normal(gen, C))).to(torch.bfloat16)
        for name, r, c in (("rows", R, C), ("cols", C, R)):
            if case["along"] in (name, "both"):
                s["q_" + name], s["sf_" + name] = u8(r, -(-c // 32) * 16), u8(-(-r // 128) * -(-c // (4 * GROUP[fmt])) * 512)
                s["y_" + name] = new(r, c, dt=torch.bfloat16)
        if own:
            import fp8_mixed_precision_saturating_gb300 as g
            s["state"] = g.TensorState(16) if case["scaling"] == "current" else None
    elif case["op"] == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["sfa"], s["da"] = _operand(gen, case["fmt"], M, K, 1.0)
        s["B"], s["sfb"], s["db"] = _operand(gen, case["fmt"], N, K, 0.02)
        s["C"] = new(M, -(-N // 8) * 8, dt=DT[case["out"]])
    else:
        T, D = case["T"], case["D"]
        sd, bd = DT[case["stream"]], DT[case["block"]]
        o = _normal(gen, T, D) * 0.7 + 0.1
        r = _normal(gen, T, D) * torch.exp(0.3 * _normal(gen, D))
        s["r"], s["o"] = r.to(sd), o.to(bd)
        G = -(-T // case["gate_rows"]) if case["gate_rows"] else 0
        s["gate"] = (0.5 + 0.3 * _normal(gen, G, D)).to(bd) if G else None
        for k in ("post", "pre"):
            s["w_" + k] = 1 + 0.2 * _normal(gen, D) if case[k] != "none" else None
            s["b_" + k] = 0.1 * _normal(gen, D) if case[k] == "layer" else None
        s["scale"] = torch.full((1,), 0.9, device="cuda") if case["alpha"] else None
        s["stat_post"], s["stat_pre"] = new(T, 2), new(T, 2)
        if case["op"] == "norm_fwd":
            s["r_out"] = new(T, D, dt=sd)
            if case["emit"]:
                fmt, N = case["emit"], case["N"]
                s["W"], s["sfw"], s["dw"] = _operand(gen, fmt, N, D, 0.02)
                s["hq"], s["hsf"] = u8(T, -(-D // 32) * 16), u8(-(-T // 128) * -(-D // (4 * GROUP[fmt])) * 512)
                s["y"] = new(T, -(-N // 8) * 8, dt=bd)
            else:
                s["h"] = new(T, D, dt=bd)
        else:
            rn = _mid(s, s["o"].float(), _stat(s["o"].float(), case["post"]))
            s["r_out"] = rn.to(sd)
            s["stat_post"], s["stat_pre"] = _stat(s["o"].float(), case["post"]), _stat(s["r_out"].float(), case["pre"])
            s["dh"], s["dr_out"] = (0.01 * _normal(gen, T, D)).to(bd), (0.01 * _normal(gen, T, D) + 1e-3).to(sd)
            s["dr"], s["do"] = new(T, D, dt=sd), new(T, D, dt=bd)
            for k in ("post", "pre"):
                s["dw_" + k] = new(D) if case[k] != "none" else None
                s["db_" + k] = new(D) if case[k] == "layer" else None
            s["dgate"] = new(G, D) if G else None
            s["dscale"] = new(1) if case["alpha"] else None
        if own:
            _plan(s)
    return s


def _plan(s):
    """The argument block a user's program keeps for a layer's norm."""
    import fp8_mixed_precision_saturating_gb300 as g
    kind = {"none": g.FP8_NORM_NONE, "rms": g.FP8_NORM_RMS, "layer": g.FP8_NORM_LAYER}
    dt = {"bf16": g.FP8_DT_BF16, "f32": g.FP8_DT_F32}
    more = {}
    if s["op"] == "norm_fwd" and s["emit"]:
        more = dict(hq=s["hq"], hsf=s["hsf"], h_fmt={"nv": g.FP4_NVFP4, "mx": g.FP4_MXFP4}[s["emit"]])
    s["plan"] = g.block_norm(
        s["T"], s["D"], dt[s["stream"]], dt[s["block"]], post=kind[s["post"]], pre=kind[s["pre"]], eps=EPS, r=s["r"], o=s["o"], gate=s["gate"],
        gate_rows=s["gate_rows"], res_scale=s["scale"], w_post=s["w_post"], b_post=s["b_post"], w_pre=s["w_pre"], b_pre=s["b_pre"], r_out=s["r_out"],
        h=s.get("h"), stat_post=s["stat_post"], stat_pre=s["stat_pre"], **more)
    if s["op"] == "norm_bwd":
        s["back"] = g.block_norm_grad(
            dh=s["dh"], dr_out=s["dr_out"], dr=s["dr"], do=s["do"], dgate=s["dgate"], dres_scale=s["dscale"], dw_post=s["dw_post"], db_post=s["db_post"],
            dw_pre=s["dw_pre"], db_pre=s["db_pre"])
        n = g.fp8_block_norm_bwd_workspace_bytes(s["plan"], s["back"])
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _stat(x, kind):
    """[T, 2]: the mean and 1 / root of a norm's rows (mean 0 for the root mean square)."""
    if kind == "none":
        return torch.stack([torch.zeros_like(x[:, 0]), torch.ones_like(x[:, 0])], dim=1)
    mean = x.sum(dim=1) / x.shape[1] if kind == "layer" else torch.zeros_like(x[:, 0])
    z = x - mean.unsqueeze(1)
    return torch.stack([mean, 1.0 / torch.sqrt((z * z).sum(dim=1) / x.shape[1] + EPS)], dim=1)


def _norm(x, stat, w, b):
    y = (x - stat[:, :1]) * stat[:, 1:]
    y = y if w is None else y * w
    return y if b is None else y + b


def _gate(s):
    if s["gate"] is None:
        return None
    return s["gate"].float()[torch.arange(s["T"], device="cuda") // s["gate_rows"]]


def _mid(s, o, stat):
    n, gate = _norm(o, stat, s["w_post"], s["b_post"]), _gate(s)
    n = n if gate is None else gate * n
    r = s["r"].float()
    return (r if s["scale"] is None else r * s["scale"]) + n


def _plain_quantize(s):
    out = {}
    x = s["x"].float()
    scale, inv = _tensor_scale(x, s["scaling"])
    for name in ("rows", "cols"):
        if s["along"] in (name, "both"):
            v = x if name == "rows" else x.t()
            q, c = _quantize(v, s["fmt"], scale)
            out[name] = ((q * c.unsqueeze(2)).view(v.shape[0], -1)[:, : v.shape[1]] * inv).to(torch.bfloat16)
    return out


def _plain_mm(s):
    a, b = _unpack(s["A"], s["sfa"], s["fmt"], s["M"], s["K"]), _unpack(s["B"], s["sfb"], s["fmt"], s["N"], s["K"])
    c = a @ b.t()
    return (c * (s["da"] * s["db"]) if s["scaled"] else c).to(DT[s["out"]])


def _plain_norm_fwd(s):
    o = s["o"].float()
    post = _stat(o, s["post"])
    r = _mid(s, o, post)
    pre = _stat(r, s["pre"])
    h = _norm(r, pre, s["w_pre"], s["b_pre"])
    out = {"r": r.to(DT[s["stream"]]), "stat_pre": pre}
    if s["post"] != "none":
        out["stat_post"] = post
    if s["emit"]:
        q, c = _quantize(h, s["emit"], torch.ones(1, device="cuda"))
        w = _unpack(s["W"], s["sfw"], s["emit"], s["N"], s["D"])
        out["y"] = (((q * c.unsqueeze(2)).view(s["T"], -1)[:, : s["D"]] @ w.t()) * s["dw"]).to(DT[s["block"]])
    else:
        out["h"] = h.to(DT[s["block"]])
    return out


def _norm_back(dy, x, stat, w, kind):
    """Gradients of a norm: of its input, its weight and its bias."""
    if kind == "none":
        return dy, None, None
    z = (x - stat[:, :1]) * stat[:, 1:]
    dz = dy * w
    dx = dz - z * ((dz * z).sum(dim=1, keepdim=True) / x.shape[1])
    if kind == "layer":
        dx = dx - dz.sum(dim=1, keepdim=True) / x.shape[1]
    return dx * stat[:, 1:], (dy * z).sum(dim=0), dy.sum(dim=0) if kind == "layer" else None


def _plain_norm_bwd(s):
    o, out = s["o"].float(), {}
    dx, dw, db = _norm_back(s["dh"].float(), s["r_out"].float(), s["stat_pre"], s["w_pre"], s["pre"])
    g = s["dr_out"].float() + dx
    out.update(dr=(g if s["scale"] is None else g * s["scale"]).to(DT[s["stream"]]), dw_pre=dw)
    if db is not None:
        out["db_pre"] = db
    if s["scale"] is not None:
        out["dscale"] = (g * s["r"].float()).sum().view(1)
    gate = _gate(s)
    if gate is not None:
        dg = g * _norm(o, s["stat_post"], s["w_post"], s["b_post"])
        where = torch.arange(s["T"], device="cuda") // s["gate_rows"]
        out["dgate"] = torch.zeros_like(s["gate"], dtype=torch.float32).index_add_(0, where, dg) if s["gate"].shape[0] > 1 else dg.sum(dim=0, keepdim=True)
    do, dw, db = _norm_back(g if gate is None else g * gate, o, s["stat_post"], s["w_post"], s["post"])
    out["do"] = do.to(DT[s["block"]])
    if dw is not None:
        out["dw_post"] = dw
    if db is not None:
        out["db_post"] = db
    return out


def _own_quantize(s):
    import fp8_mixed_precision_saturating_gb300 as g
    fmt = g.FP4_NVFP4 if s["fmt"] == "nv" else g.FP4_MXFP4
    R, C, st = s["rows"], s["cols"], s["state"]
    g.fp4_quantize(s["x"], R, C, C, fmt, g.FP8_SCALE_CURRENT, st, s.get("q_rows"), s.get("sf_rows"), s.get("q_cols"), s.get("sf_cols"))
    out = {}
    for name, r, c in (("rows", R, C), ("cols", C, R)):
        if s["along"] in (name, "both"):
            g.fp4_dequantize(s["q_" + name], s["sf_" + name], r, c, fmt, st and st.scale_inv, s["y_" + name], g.FP8_DT_BF16, c)
            out[name] = s["y_" + name]
    return out


def _own_mm(s):
    import fp8_mixed_precision_saturating_gb300 as g
    da, db = (s["da"], s["db"]) if s["scaled"] else (None, None)
    g.fp4_scaled_mm(s["A"], s["sfa"], s["B"], s["sfb"], s["M"], s["N"], s["K"], g.FP4_NVFP4 if s["fmt"] == "nv" else g.FP4_MXFP4, da, db, s["C"],
                    g.FP8_DT_BF16 if s["out"] == "bf16" else g.FP8_DT_F32, s["C"].shape[1])
    return s["C"][:, : s["N"]]


def _own_norm_fwd(s):
    import fp8_mixed_precision_saturating_gb300 as g
    g.fp8_block_norm_fwd(s["plan"])
    out = {"r": s["r_out"], "stat_pre": s["stat_pre"]}
    if s["post"] != "none":
        out["stat_post"] = s["stat_post"]
    if s["emit"]:
        g.fp4_scaled_mm(s["hq"], s["hsf"], s["W"], s["sfw"], s["T"], s["N"], s["D"], g.FP4_NVFP4 if s["emit"] == "nv" else g.FP4_MXFP4, None, s["dw"],
                        s["y"], g.FP8_DT_BF16 if s["block"] == "bf16" else g.FP8_DT_F32, s["y"].shape[1])
        out["y"] = s["y"][:, : s["N"]]
    else:
        out["h"] = s["h"]
    return out


def _own_norm_bwd(s):
    import fp8_mixed_precision_saturating_gb300 as g
    g.fp8_block_norm_bwd(s["plan"], s["back"], s["ws"], s["ws"].numel())
    names = ("dr", "do", "dw_pre", "db_pre", "dw_post", "db_post", "dgate", "dscale")
    return {k: s[k] for k in names if s[k] is not None}


_plain = {"quantize": _plain_quantize, "mm": _plain_mm, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}
_own = {"quantize": _own_quantize, "mm": _own_mm, "norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def _bytes4(fmt, r, c):
    return r * c * 0.5 + r * -(-c // GROUP[fmt])


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        ways = [(R, C)] * (case["along"] != "cols") + [(C, R)] * (case["along"] != "rows")
        return {"bytes": 2 * R * C + sum(_bytes4(case["fmt"], r, c) + 2 * r * c for r, c in ways), "flops": 4 * R * C * len(ways)}
    if case["op"] == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _bytes4(case["fmt"], M, K) + _bytes4(case["fmt"], N, K) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    T, D, sb, bb = case["T"], case["D"], size[case["stream"]], size[case["block"]]
    G = -(-T // case["gate_rows"]) if case["gate_rows"] else 0
    n, par = T * D, 4 * D * sum({"none": 0, "rms": 1, "layer": 2}[case[k]] for k in ("post", "pre")) + G * D * bb
    if case["op"] == "norm_fwd":
        out = T * case["N"] * bb + _bytes4(case["emit"], case["N"], D) + _bytes4(case["emit"], T, D) if case["emit"] else n * bb
        return {"bytes": 2 * n * sb + n * bb + par + 16 * T + out, "flops": 12 * n + 2 * n * case["N"]}
    # r is read for its scale's gradient, the norms' inputs again, four gradients in and out
    return {"bytes": n * (3 * sb + 3 * bb + (sb if case["alpha"] else 0)) + 2 * par + 16 * T, "flops": 24 * n}


# ------------------------------------------------------------------------------------------------
# in 64 bits, from the definitions
# ------------------------------------------------------------------------------------------------
def _nearest(v, table):
    """Nearest of a sorted table of magnitudes by the midpoints between them, ties to the even place, v's sign kept."""
    mids = (table[1:] + table[:-1]) / 2
    a = v.abs().contiguous()
    low, high = torch.bucketize(a, mids), torch.bucketize(a, mids, right=True)
    return table[torch.where(low % 2 == 0, low, high)] * torch.sign(v)


def _rounded64(v, fmt, d):
    """v [R, C] in 64 bits -> the values that its 4-bit form stands for; d: the tensor's scale."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    R, C = v.shape
    g = GROUP[fmt]
    z = torch.zeros(R, -(-C // g) * g, dtype=torch.float64, device=v.device)
    z[:, :C] = v
    z = z.reshape(-1, g)
    top = z.abs().max(dim=1, keepdim=True).values
    if fmt == "nv":
        grid = sorted({m * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8, 16)} | {m * 2.0 ** -9 for m in range(8)})
        grid = torch.tensor([x for x in grid if x <= 448], dtype=torch.float64, device=v.device)
        unit = _nearest(top / (6 * d), grid) * d
    else:
        powers = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device=v.device)
        unit = torch.where(top > 0, powers[torch.bucketize(top, 6 * powers)], torch.ones_like(top))
    y = torch.where(unit > 0, _nearest(z / torch.where(unit > 0, unit, torch.ones_like(unit)), mags) * unit, torch.zeros_like(z))
    return y.reshape(R, -1)[:, :C]


def _decoded64(codes, atoms, fmt, R, C):
    """A stored 4-bit operand as numbers in 64 bits, element by element from its bytes' places."""
    k = torch.arange(C, device=codes.device)
    nib = (codes[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
    expo, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(expo == 0, man * 0.5, torch.ldexp(1 + man * 0.5, expo - 1))
    row, grp = torch.arange(R, device=codes.device).view(-1, 1), (k // GROUP[fmt]).view(1, -1)
    na = -(-(-(-C // GROUP[fmt])) // 4)
    b = atoms[((row // 128) * na + grp // 4) * 512 + 16 * (row % 32) + 4 * ((row // 32) % 4) + grp % 4].int()
    if fmt == "nv":
        e, m = (b >> 3) & 15, (b & 7).double()
        scale = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(8 + m, e - 10))
    else:
        scale = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
    return torch.where(nib >= 8, -mag, mag) * scale


def exact(case, seed):
    with torch.enable_grad():
        return _exact(case, prepare(case, seed))


def _exact(case, s):
    if case["op"] == "quantize":
        x = s["x"].double()
        d = x.abs().max() / 2688 if case["scaling"] == "current" else torch.ones((), dtype=torch.float64, device=x.device)
        return {k: _rounded64(x if k == "rows" else x.t(), case["fmt"], d) for k in ("rows", "cols") if case["along"] in (k, "both")}
    if case["op"] == "mm":
        c = torch.matmul(_decoded64(s["A"], s["sfa"], case["fmt"], case["M"], case["K"]), _decoded64(s["B"], s["sfb"], case["fmt"], case["N"], case["K"]).T)
        return c * (s["da"].double() * s["db"].double()) if case["scaled"] else c

    def leaf(name):
        return None if s[name] is None else s[name].double().requires_grad_(case["op"] == "norm_bwd")

    def norm(x, kind, w, b):
        if kind == "none":
            return x, None
        mean = x.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
        root = ((x - mean).pow(2).mean(dim=1, keepdim=True) + EPS).rsqrt()
        y = (x - mean) * root * w
        return (y if b is None else y + b), torch.cat([mean, root], dim=1)

    v = {k: leaf(k) for k in ("r", "o", "gate", "w_post", "b_post", "w_pre", "b_pre", "scale")}
    n, post = norm(v["o"], case["post"], v["w_post"], v["b_post"])
    if v["gate"] is not None:
        n = n * v["gate"].repeat_interleave(min(case["gate_rows"], case["T"]), dim=0)[: case["T"]]
    mid = n + (v["r"] if v["scale"] is None else v["r"] * v["scale"])
    if case["op"] == "norm_fwd":
        h, pre = norm(mid, case["pre"], v["w_pre"], v["b_pre"])
        out = {"r": mid, "stat_pre": pre}
        if post is not None:
            out["stat_post"] = post
        if not case["emit"]:
            out["h"] = h
            return out
        one = torch.ones((), dtype=torch.float64, device=h.device)
        w = _decoded64(s["W"], s["sfw"], case["emit"], case["N"], case["D"])
        out["y"] = torch.matmul(_rounded64(h, case["emit"], one), w.T) * s["dw"].double()
        return out
    # two pieces, as the backward sees them: the next norm reads the stored stream, the block's side its own input
    stored = s["r_out"].double().requires_grad_(True)
    h, _ = norm(stored, case["pre"], v["w_pre"], v["b_pre"])
    names = [k for k in ("w_pre", "b_pre") if v[k] is not None]
    first = dict(zip(["stored"] + names, torch.autograd.grad(h, [stored] + [v[k] for k in names], s["dh"].double())))
    g = first["stored"] + s["dr_out"].double()
    names = [k for k in ("r", "o", "gate", "w_post", "b_post", "scale") if v[k] is not None]
    second = dict(zip(names, torch.autograd.grad(mid, [v[k] for k in names], g)))
    out = {"dr": second["r"], "do": second["o"], "dw_pre": first["w_pre"]}
    for name, key in (("db_pre", "b_pre"), ("dw_post", "w_post"), ("db_post", "b_post"), ("dgate", "gate"), ("dscale", "scale")):
        if v[key] is not None:
            out[name] = (first if key in first else second)[key]
    return out
