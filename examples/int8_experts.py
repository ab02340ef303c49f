"""An expert block served in 8-bit integers, its router included: router product -> choice of experts -> choices sorted by
expert -> gather and quantise -> gate and up products -> SwiGLU and quantise -> down products -> weighted sum, plus the input.

    python examples/int8_experts.py [--tokens T] [--experts E] [--groups G] [--top-k K] [--hidden H] [--inner I]

Weights have a scale per output channel, activations a scale per token. All steps are enqueued on the current stream; nothing
is copied to the host, so a block can be captured into a graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_bf16_amd as qg  # noqa: E402

W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)


class Codes:
    """rows x cols in int8 at a pitch of 16 bytes, with a scale per row."""

    def __init__(self, rows, cols):
        self.rows, self.cols = rows, cols
        self.q = torch.empty(rows, -(-cols // 16) * 16, device="cuda", dtype=torch.int8)
        self.s = torch.empty(rows, device="cuda")

    def layouts(self, rows=None, **kw):
        rows, pitch = rows or self.rows, self.q.stride(0)
        stride = {"stride": rows} if "num" in kw and "offsets" not in kw else {}
        return (qg.layout("i8", rows, self.cols, ld=pitch, **kw, **({"stride": rows * pitch} if stride else {})),
                qg.layout("f32", rows, 1, **kw, **stride))

    def fill(self, engine, x, act=qg.MX_IDENTITY, rows=None):
        qd, sd = self.layouts()
        engine.int_quantize(x, qg.layout("bf16", x.shape[0], x.shape[1], ld=x.stride(0)), self.q, qd, self.s, sd, act=act, rows=rows)
        return self


class ExpertBlock:
    """router: E x H, gate_up: E x 2I x H, down: E x H x I, bfloat16 (the experts are quantised once); bias: E fp32 for balance.
    Sizes are multiples of 8."""

    def __init__(self, engine, router, bias, gate_up, down, tokens, routing):
        self.engine, self.space, self.routing = engine, qg.workspace(), routing
        self.router, self.bias = router, bias
        self.experts, self.hidden, self.inner = down.shape
        self.tokens, self.top_k = tokens, routing.top_k
        rows = tokens * self.top_k
        self.w1 = Codes(self.experts * 2 * self.inner, self.hidden).fill(engine, gate_up.flatten(0, 1))
        self.w2 = Codes(self.experts * self.hidden, self.inner).fill(engine, down.flatten(0, 1))
        self.x, self.h = Codes(rows, self.hidden), Codes(rows, self.inner)
        self.logits = torch.empty(tokens, self.experts, device="cuda")
        self.ids, self.rows, self.back = (torch.empty(rows, device="cuda", dtype=torch.int32) for _ in range(3))
        self.weights = torch.empty(rows, device="cuda")
        self.offsets = torch.empty(self.experts + 1, device="cuda", dtype=torch.int32)
        self.gate_up = torch.empty(rows, 2 * self.inner, device="cuda", dtype=torch.bfloat16)
        self.out = torch.empty(rows, self.hidden, device="cuda", dtype=torch.bfloat16)
        self.op = qg.operation(quant_a=W8A8, quant_b=W8A8)

    def product(self, a, w, d):
        off = self.offsets.data_ptr()
        (ad, ud), (bd, vd) = a.layouts(num=self.experts, offsets=off), w.layouts(w.rows // self.experts, num=self.experts)
        dd = qg.layout("bf16", *d.shape, num=self.experts, offsets=off)
        self.engine.run(self.op, 1.0, a.q, ad, a.s, ud, w.q, bd, w.s, vd, 0.0, None, None, d, dd, self.space.desc)

    def __call__(self, x):
        """x: tokens x H bfloat16, rows at any pitch of 16 bytes; returns x plus its experts' weighted sum."""
        g, t = self.engine, self.tokens
        xd, yd, ld = qg.layout("bf16", t, self.hidden, ld=x.stride(0)), qg.layout("bf16", t, self.hidden), qg.layout("f32", t, self.experts)
        kd, wd = qg.layout("i32", t, self.top_k), qg.layout("f32", t, self.top_k)
        g.run(qg.operation(), 1.0, x, xd, None, None, self.router, qg.layout("bf16", self.experts, self.hidden), None, None,
              0.0, None, None, self.logits, ld, self.space.desc)
        g.route(self.routing, self.logits, ld, self.bias, self.ids, kd, self.weights, wd)
        g.group_rows(self.experts, self.ids, kd, self.offsets, self.rows, self.back, self.space.desc)
        self.x.fill(g, x, rows=self.rows)
        self.product(self.x, self.w1, self.gate_up)
        self.h.fill(g, self.gate_up, act=qg.MX_SWIGLU)
        self.product(self.h, self.w2, self.out)
        y = torch.empty(t, self.hidden, device="cuda", dtype=torch.bfloat16)
        g.combine(self.out, qg.layout("bf16", *self.out.shape), self.back, self.weights, wd, y, yd, beta=1.0, C=x, Cd=xd)
        return y


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    a = ap.parse_args()
    torch.manual_seed(0)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    router = torch.randn(a.experts, a.hidden, **bf) * 0.02
    w1 = torch.randn(a.experts, 2 * a.inner, a.hidden, **bf) * 0.02
    w2 = torch.randn(a.experts, a.hidden, a.inner, **bf) * 0.02
    routing = qg.routing(qg.ROUTE_SIGMOID, a.top_k, groups=a.groups, top_groups=max(1, a.groups // 2), group_best=2, renormalize=True)
    block = ExpertBlock(qg.Gemm(), router, torch.zeros(a.experts, device="cuda"), w1, w2, a.tokens, routing)
    x = torch.randn(a.tokens, a.hidden, **bf)
    for _ in range(3):
        y = block(x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        y = block(x)
    end.record()
    torch.cuda.synchronize()
    flop = 6 * a.tokens * a.top_k * a.hidden * a.inner
    ms = begin.elapsed_time(end) / 10
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, {a.top_k} each: {ms:.3f} ms, "
          f"{flop / ms / 1e9:.0f} TOP/s, output rms {y.float().pow(2).mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
