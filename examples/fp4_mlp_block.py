"""An MLP block in 4 bits between two norms: a training step's forward and backward, and one token.

    python examples/fp4_mlp_block.py            (needs a GB300 and the built library)

The residual stream r stays in bf16. Each call of the norms does what stands between two blocks in one pass: the norm
after the last block with its gate, the scaled residual, and the norm before the next block, whose output goes straight
into the 4-bit operand that the next projection reads. The weights are kept in bf16 and re-quantised after an optimizer
step (both ways: the forward contracts them along their rows, the data gradient down their columns)."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_mixed_precision_saturating_gb300 as g  # noqa: E402

BF16, F32 = g.FP8_DT_BF16, g.FP8_DT_F32


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Operand:
    """A 4-bit operand's buffers: MN rows along a contraction of K."""

    def __init__(self, mn, k, fmt):
        self.mn, self.k, self.fmt = mn, k, fmt
        self.q = empty(mn, g.fp4_row_bytes(k), dtype=torch.uint8)
        self.sf = empty(g.fp4_scale_bytes(fmt, mn, k), dtype=torch.uint8)


def quantize(x, rows=None, cols=None, state=None):
    """x [R, C] into `rows` (along its rows) and / or `cols` (down its columns)."""
    fmt = (rows or cols).fmt
    g.fp4_quantize(x, x.shape[0], x.shape[1], x.stride(0), fmt, g.FP8_SCALE_CURRENT, state, rows and rows.q, rows and rows.sf, cols and cols.q, cols and cols.sf)


def product(a, b, out, da=None, db=None):
    """out [M, N] = a b^T of two operands."""
    g.fp4_scaled_mm(a.q, a.sf, b.q, b.sf, a.mn, b.mn, a.k, a.fmt, da, db, out, F32 if out.dtype == torch.float32 else BF16, out.stride(0))


class Block:
    """y = relu(h W_up)^2 W_down between the norms, for `tokens` tokens."""

    def __init__(self, tokens, width, hidden, fmt=g.FP4_NVFP4, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.T, self.D, self.H, self.fmt = tokens, width, hidden, fmt
        self.w_up, self.w_down = (n(width, hidden) * width ** -0.5).bfloat16(), (n(hidden, width) * hidden ** -0.5).bfloat16()
        self.w_post, self.w_pre, self.gate = 1 + 0.1 * n(width), 1 + 0.1 * n(width), (0.5 + 0.1 * n(1, width)).bfloat16()
        self.alpha = torch.full((1,), 0.95, device="cuda")
        # 4-bit weights, both ways, each with a scale for the tensor (NVFP4)
        nv = fmt == g.FP4_NVFP4
        self.up, self.up_t, self.up_s = Operand(hidden, width, fmt), Operand(width, hidden, fmt), g.TensorState() if nv else None
        self.down, self.down_t, self.down_s = Operand(width, hidden, fmt), Operand(hidden, width, fmt), g.TensorState() if nv else None
        self.refresh()
        # what the forward leaves for the backward
        self.h, self.hq = empty(tokens, width), Operand(tokens, width, fmt)
        self.a, self.act, self.actq = empty(tokens, hidden), empty(tokens, hidden), Operand(tokens, hidden, fmt)
        self.o, self.r_in, self.r_out, self.h_out = empty(tokens, width), empty(tokens, width), empty(tokens, width), empty(tokens, width)
        self.stats = [empty(tokens, 2, dtype=torch.float32) for _ in range(3)]

    def refresh(self):
        """The 4-bit weights after an optimizer step: W [K, N] down its columns for the forward, along its rows for the data gradient."""
        quantize(self.w_up, self.up_t, self.up, self.up_s)
        quantize(self.w_down, self.down_t, self.down, self.down_s)

    def inv(self, state):
        return None if state is None else state.scale_inv

    def forward(self, r):
        """(the stream behind the block, the next block's input)"""
        T, D = self.T, self.D
        self.r_in.copy_(r)
        self.before = g.block_norm(T, D, BF16, BF16, pre=g.FP8_NORM_RMS, r=self.r_in, w_pre=self.w_pre, h=self.h, stat_pre=self.stats[0], hq=self.hq.q,
                                   hsf=self.hq.sf, h_fmt=self.fmt)
        g.fp8_block_norm_fwd(self.before)
        product(self.hq, self.up, self.a, None, self.inv(self.up_s))
        torch.square(torch.relu(self.a), out=self.act)
        quantize(self.act, self.actq)
        product(self.actq, self.down, self.o, None, self.inv(self.down_s))
        self.after = g.block_norm(T, D, BF16, BF16, post=g.FP8_NORM_RMS, pre=g.FP8_NORM_RMS, r=self.r_in, o=self.o, gate=self.gate, gate_rows=T,
                                  res_scale=self.alpha, w_post=self.w_post, w_pre=self.w_pre, r_out=self.r_out, h=self.h_out, stat_post=self.stats[1],
                                  stat_pre=self.stats[2])
        g.fp8_block_norm_fwd(self.after)
        return self.r_out, self.h_out

    def backward(self, dr_out, dh_out):
        """The gradients of the stream, the weights, the norms' weights, the gate and the residual's scale."""
        T, D, H, fmt = self.T, self.D, self.H, self.fmt
        vec = lambda *s: empty(*s, dtype=torch.float32)  # noqa: E731
        out = {"dr": empty(T, D), "dgate": vec(1, D), "dalpha": vec(1), "dw_post": vec(D), "dw_pre": vec(D), "dw_up": vec(D, H), "dw_down": vec(H, D)}
        do, first = empty(T, D), vec(D)

        def norm_back(f, **kw):
            b = g.block_norm_grad(**kw)
            n = g.fp8_block_norm_bwd_workspace_bytes(f, b)
            g.fp8_block_norm_bwd(f, b, empty(max(n, 16), dtype=torch.uint8), n)

        norm_back(self.after, dh=dh_out, dr_out=dr_out, dr=out["dr"], do=do, dgate=out["dgate"], dres_scale=out["dalpha"], dw_post=out["dw_post"], dw_pre=out["dw_pre"])
        # the block's own backward: every gradient along the rows for dgrad and down the columns for wgrad
        do_r, do_c, act_c = Operand(T, D, fmt), Operand(D, T, fmt), Operand(H, T, fmt)
        quantize(do, do_r, do_c)
        quantize(self.act, cols=act_c)
        da = empty(T, H)
        product(do_r, self.down_t, da, None, self.inv(self.down_s))
        product(act_c, do_c, out["dw_down"])
        da.mul_(torch.relu(self.a).mul_(2))
        da_r, da_c, h_c = Operand(T, H, fmt), Operand(H, T, fmt), Operand(D, T, fmt)
        quantize(da, da_r, da_c)
        quantize(self.h, cols=h_c)
        dh = empty(T, D)
        product(da_r, self.up_t, dh, None, self.inv(self.up_s))
        product(h_c, da_c, out["dw_up"])
        # the norm before the block: its stream is r itself, and the gradient joins the one around the block
        self.before.r_out, self.before.ld_r_out = self.r_in.data_ptr(), self.r_in.stride(0)
        norm_back(self.before, dh=dh, dr_out=out["dr"], dr=out["dr"], dw_pre=first)
        self.before.r_out = None
        out["dw_pre"] += first
        return out


def reference(block, r, dr_out, dh_out):
    """The same block in fp32 without any rounding, by autograd."""
    p = {k: getattr(block, k).float().requires_grad_() for k in ("w_up", "w_down", "w_post", "w_pre", "gate", "alpha")}
    x = r.float().requires_grad_()
    norm = lambda v, w: v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + 1e-5) * w  # noqa: E731
    o = torch.relu(norm(x, p["w_pre"]) @ p["w_up"]).square() @ p["w_down"]
    r_out = p["alpha"] * x + p["gate"] * norm(o, p["w_post"])
    h_out = norm(r_out, p["w_pre"])
    ((r_out * dr_out.float()).sum() + (h_out * dh_out.float()).sum()).backward()
    return r_out, h_out, {"dr": x.grad, "dgate": p["gate"].grad, "dalpha": p["alpha"].grad, "dw_post": p["w_post"].grad, "dw_pre": p["w_pre"].grad,
                          "dw_up": p["w_up"].grad, "dw_down": p["w_down"].grad}


def cosine(a, b):
    a, b = a.detach().double().reshape(-1), b.detach().double().reshape(-1)
    return float(a @ b / (a.norm() * b.norm()))


def main():
    torch.manual_seed(0)
    found = {}
    for name, fmt in (("NVFP4", g.FP4_NVFP4), ("MXFP4", g.FP4_MXFP4)):
        for tokens in (2048, 1):
            block = Block(tokens, 1536, 6144, fmt)
            r = torch.randn(tokens, 1536, device="cuda").bfloat16()
            dr, dh = torch.randn_like(r) * 0.1, torch.randn_like(r) * 0.1
            r_out, h_out = block.forward(r)
            grads = block.backward(dr, dh) if tokens > 1 else {}
            torch.cuda.synchronize()
            g.fp8_poll_device_error()
            want_r, want_h, want = reference(block, r, dr, dh)
            found[name, tokens] = {"r": cosine(r_out, want_r), "h": cosine(h_out, want_h), **{k: cosine(v, want[k]) for k, v in grads.items()}}
            print(f"{name}, {tokens} tokens, cosine with the block in fp32:", ", ".join(f"{k} {v:.4f}" for k, v in found[name, tokens].items()))
    return found


if __name__ == "__main__":
    main()
