"""The 4-bit and block-norm calls captured in a CUDA graph, from the first call of a process on, and from several threads and streams
at once: the bits of the same calls made eagerly, one after the other."""
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Work:
    """Buffers of one run of every call: x in 4 bits both ways and back, products that take each kernel, norms and gradients."""

    def __init__(self, g, fmt, T, D, N, seed):
        gen = torch.Generator("cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        u8 = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")  # noqa: E731
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.g, self.fmt, self.T, self.D, self.N = g, fmt, T, D, N
        self.x, self.w = n(T, D).bfloat16(), n(N, D).bfloat16()
        op = lambda r, c: (u8(r * g.fp4_row_bytes(c)), u8(g.fp4_scale_bytes(fmt, r, c)))  # noqa: E731
        self.xr, self.xc, self.wr, self.hr = op(T, D), op(D, T), op(N, D), op(T, D)
        self.sx = g.TensorState() if fmt == g.FP4_NVFP4 else None
        self.y, self.back, self.y1, self.dw = e(T, N), e(T, D), e(1, N), e(D, D, dt=torch.float32)
        self.o, self.gate, self.par, self.alpha = n(T, D).bfloat16(), n(1, D).bfloat16(), n(D), torch.full((1,), 0.9, device="cuda")
        self.r_out, self.h, self.st = e(T, D), e(T, D), (e(T, 2, dt=torch.float32), e(T, 2, dt=torch.float32))
        self.f = g.block_norm(T, D, g.FP8_DT_BF16, g.FP8_DT_BF16, post=g.FP8_NORM_RMS, pre=g.FP8_NORM_LAYER, r=self.x, o=self.o, gate=self.gate, gate_rows=T,
                              res_scale=self.alpha, w_post=self.par, w_pre=self.par, b_pre=self.par, r_out=self.r_out, h=self.h, hq=self.hr[0], hsf=self.hr[1],
                              h_fmt=fmt, stat_post=self.st[0], stat_pre=self.st[1])
        self.dx, self.do, self.sums = e(T, D), e(T, D), [e(D, dt=torch.float32) for _ in range(4)]
        self.b = g.block_norm_grad(dh=self.h, dr_out=self.r_out, dr=self.dx, do=self.do, dw_post=self.sums[0], dw_pre=self.sums[1], db_pre=self.sums[2], dgate=self.sums[3])
        self.n = g.fp8_block_norm_bwd_workspace_bytes(self.f, self.b)
        self.ws = u8(self.n)

    def calls(self):
        g, T, D, N, fmt = self.g, self.T, self.D, self.N, self.fmt
        g.fp4_quantize(self.x, T, D, D, fmt, g.FP8_SCALE_CURRENT, self.sx, *self.xr, *self.xc)
        g.fp4_quantize(self.w, N, D, D, fmt, g.FP8_SCALE_CURRENT, None, *self.wr)
        d = self.sx and self.sx.scale_inv
        g.fp4_dequantize(*self.xr, T, D, fmt, d, self.back, g.FP8_DT_BF16, D)
        g.fp4_scaled_mm(*self.xr, *self.wr, T, N, D, fmt, d, None, self.y, g.FP8_DT_BF16, N)
        g.fp4_scaled_mm(*self.xr, *self.wr, 1, N, D, fmt, d, None, self.y1, g.FP8_DT_BF16, N)
        g.fp4_scaled_mm(*self.xc, *self.xc, D, D, T, fmt, d, d, self.dw, g.FP8_DT_F32, D)
        g.fp8_block_norm_fwd(self.f)
        g.fp8_block_norm_bwd(self.f, self.b, self.ws, self.n)

    def results(self):
        return [*self.xr, *self.xc, *self.wr, self.back, self.y, self.y1, self.dw, self.r_out, self.h, *self.hr, *self.st, self.dx, self.do, *self.sums]

    def clear(self):
        for t in self.results():
            t.zero_()


def eager(w):
    w.clear()
    w.calls()
    torch.cuda.synchronize()
    return [t.clone() for t in w.results()]


def capture_first():
    """(in a process of its own) The calls are captured before any of them has been made."""
    sys.path.insert(0, ROOT)
    import fp8_mixed_precision_saturating_gb300 as g
    for fmt, T, D, N in ((g.FP4_NVFP4, 300, 1024, 512), (g.FP4_MXFP4, 1300, 1024, 2048)):
        w = Work(g, fmt, T, D, N, 1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.calls()
        w.clear()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        g.fp8_poll_device_error()
        got = [t.clone() for t in w.results()]
        assert all(torch.equal(a, b) for a, b in zip(got, eager(w)))
        assert all(t.count_nonzero() for t in got)
    print("captured")


def test_capture_from_the_first_call_on():
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path.insert(0, 'tests'); import test_gpu_fp4_graph as t; t.capture_first()"], cwd=ROOT,
                       capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_several_threads_and_streams():
    import fp8_mixed_precision_saturating_gb300 as g
    works = [Work(g, *s, seed=i) for i, s in enumerate(((g.FP4_NVFP4, 1300, 1024, 512), (g.FP4_MXFP4, 700, 2048, 256), (g.FP4_NVFP4, 64, 4096, 1024), (g.FP4_MXFP4, 1, 512, 256)))]
    want = [eager(w) for w in works]
    failed = []

    def work(w, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    w.clear()
                    w.calls()
                torch.cuda.current_stream().synchronize()
            assert all(torch.equal(a, b) for a, b in zip(w.results(), want))
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(works, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    g.fp8_poll_device_error()
