"""The 8-bit operators as a serving program uses them.

    python examples/fp8_serving.py [--tokens 4] [--d-model 1024] [--d-ff 512] [--experts 8] [--top-k 2]

Weights are quantised to e4m3 in 128 x 128 blocks once.  Then, per step: a dense projection (the
activations quantised by row, the block-scaled product with its bias and GELU) and a
mixture-of-experts layer on its result, captured into a HIP graph after the first run.  Prints how far
both are from the same step in fp32 from the unquantised weights, and the time of a replay.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_algebra_sgemm_amd as lib  # noqa: E402


def blocks(n):
    return -(-n // 128)


def quantize_weights(w):
    """e4m3 values and 128 x 128 scales of a stack of fp32 matrices (E, rows, cols), dense."""
    e, rows, cols = w.shape
    q = torch.empty((e, rows, cols), dtype=torch.uint8, device=w.device)
    s = torch.empty((e, blocks(cols), blocks(rows)), device=w.device)
    for i in range(e):
        lib.fp8_quantize(rows, cols, lib.TYPE_F32, w[i], cols, 128, q[i], cols, s[i], blocks(rows))
    return q, s


class Step:
    """A dense D x D projection with GELU, then E experts of inner size I."""

    def __init__(self, tokens, d, i, experts, top_k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, size=1.0):
            return torch.randn(shape, generator=g, device="cuda") * size
        self.wp, self.bias = normal(1, d, d, size=d ** -0.5), normal(d, size=0.1)
        self.w1 = normal(experts, 2 * i, d, size=d ** -0.5)
        self.w2 = normal(experts, d, i, size=i ** -0.5)
        self.router = normal(experts, d, size=1.5 * d ** -0.5).bfloat16()
        self.x = normal(tokens, d).bfloat16()
        self.qp, self.sp = quantize_weights(self.wp)
        self.q1, self.s1 = quantize_weights(self.w1)
        self.q2, self.s2 = quantize_weights(self.w2)
        self.shape = lib.MoeShape(tokens=tokens, d_model=d, d_ff=i, experts=experts, top_k=top_k,
                                  type=lib.TYPE_BF16, weight_type=lib.TYPE_E4M3, act=lib.ACT_SILU,
                                  gated=True, norm_topk=True)
        self.qx = torch.empty((tokens, d), dtype=torch.uint8, device="cuda")
        self.sx = torch.empty((blocks(d), tokens), device="cuda")
        self.h, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.ids = torch.empty((tokens, top_k), dtype=torch.int32, device="cuda")
        self.w = torch.empty((tokens, top_k), device="cuda")
        self.ws = torch.empty(lib.moe_ffn_workspace(self.shape), dtype=torch.uint8, device="cuda")

    def __call__(self):
        t, d, i = self.shape.tokens, self.shape.d_model, self.shape.d_ff
        lib.fp8_quantize(t, d, lib.TYPE_BF16, self.x, d, 1, self.qx, d, self.sx, t)
        lib.fp8_gemm_bias_act(t, d, d, 1.0, self.qx, d, self.sx, t, self.qp, d, self.sp, blocks(d), 128,
                              self.bias, lib.ACT_GELU_TANH, lib.TYPE_BF16, self.h, d, fast_sums=True)
        lib.moe_ffn(self.shape, self.h, d, self.router, d, self.q1, d, self.s1, self.q2, i, self.s2,
                    self.ids, self.w, self.y, d, self.ws, self.ws.numel())
        return self.y

    def in_fp32(self):
        """The same step from the unquantised weights (the experts that were chosen)."""
        h = torch.nn.functional.gelu(self.x.float() @ self.wp[0].t() + self.bias, approximate="tanh")
        y = torch.zeros_like(h)
        for t in range(h.shape[0]):
            for e, w in zip(self.ids[t].tolist(), self.w[t].tolist()):
                a, b = (self.w1[e] @ h[t]).chunk(2)
                y[t] += w * (self.w2[e] @ (torch.nn.functional.silu(a) * b))
        return h, y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4), ("d-model", 1024), ("d-ff", 512), ("experts", 8), ("top-k", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    lib.gemm_create()
    try:
        step = Step(a.tokens, a.d_model, a.d_ff, a.experts, a.top_k)
        step()
        torch.cuda.synchronize()
        h, y = step.in_fp32()
        errors = [float((got.float() - want).norm() / want.norm())
                  for got, want in ((step.h, h), (step.y, y))]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            graph.replay()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(50):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print("relative error against fp32 weights: projection %.4f, layer %.4f; %.1f us a step"
              % (errors[0], errors[1], start.elapsed_time(end) / 50 * 1e3))
        return errors
    finally:
        torch.cuda.synchronize()
        lib.gemm_destroy()


if __name__ == "__main__":
    main()
