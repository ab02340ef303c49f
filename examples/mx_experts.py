"""An expert block served in MXFP4: router choice -> choices sorted by expert -> gather and quantise -> gate and up products ->
SwiGLU and quantise -> down products -> weighted sum of each token's experts.

    python examples/mx_experts.py [--tokens T] [--experts E] [--top-k K] [--hidden H] [--inner I]

All steps are enqueued on the current stream; nothing is copied to the host, so a block can be captured into a graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_bf16_amd as qg  # noqa: E402

MX = (qg.QUANT_MX, 32, 1, 0)


def up(n, to):
    return -(-n // to) * to


class Matrix:
    """An MXFP4 operand: codes, scales, and their layouts (num > 0: that many matrices of rows x cols, one per expert)."""

    def __init__(self, rows, cols, num=0):
        self.rows, self.cols, self.num = rows, cols, num
        n = rows * max(num, 1)
        self.q = torch.empty(n, up(cols, 32) // 2, device="cuda", dtype=torch.uint8)
        self.s = torch.empty(n, up(-(-cols // 32), 16), device="cuda", dtype=torch.uint8)

    def whole(self):
        n = self.rows * max(self.num, 1)
        return qg.layout("e2m1", n, self.cols), qg.layout("e8m0", n, -(-self.cols // 32))

    def weights(self):
        blocks = -(-self.cols // 32)
        return (qg.layout("e2m1", self.rows, self.cols, num=self.num, stride=self.rows * self.q.shape[1] * 2),
                qg.layout("e8m0", self.rows, blocks, num=self.num, stride=self.rows * self.s.shape[1]))

    def grouped(self, experts, offsets):
        return (qg.layout("e2m1", self.rows, self.cols, num=experts, offsets=offsets.data_ptr()),
                qg.layout("e8m0", self.rows, -(-self.cols // 32), num=experts, offsets=offsets.data_ptr()))

    def fill(self, engine, x, act=qg.MX_IDENTITY, rows=None):
        q, s = self.whole()
        engine.mx_quantize(x, qg.layout("bf16", x.shape[0], x.shape[1], ld=x.stride(0)), self.q, q, self.s, s, act=act,
                           rows=rows)
        return self


class ExpertBlock:
    """gate_up: E x 2I x H, down: E x H x I, bfloat16; quantised once. Sizes are multiples of 8."""

    def __init__(self, engine, gate_up, down, tokens, top_k):
        self.engine, self.space = engine, qg.workspace()
        self.experts, self.hidden, self.inner = down.shape
        self.tokens, self.top_k = tokens, top_k
        rows = tokens * top_k
        self.w1 = Matrix(2 * self.inner, self.hidden, self.experts).fill(engine, gate_up.flatten(0, 1))
        self.w2 = Matrix(self.hidden, self.inner, self.experts).fill(engine, down.flatten(0, 1))
        self.x, self.h = Matrix(rows, self.hidden), Matrix(rows, self.inner)
        self.gate_up = torch.empty(rows, 2 * self.inner, device="cuda", dtype=torch.bfloat16)
        self.out = torch.empty(rows, self.hidden, device="cuda", dtype=torch.bfloat16)
        self.op = qg.operation(quant_a=MX, quant_b=MX)
        self.offsets = torch.empty(self.experts + 1, device="cuda", dtype=torch.int32)
        self.rows, self.back = (torch.empty(rows, device="cuda", dtype=torch.int32) for _ in range(2))

    def product(self, a, w, d, offsets):
        (ad, ud), (bd, vd) = a.grouped(self.experts, offsets), w.weights()
        dd = qg.layout("bf16", d.shape[0], d.shape[1], num=self.experts, offsets=offsets.data_ptr())
        self.engine.run(self.op, 1.0, a.q, ad, a.s, ud, w.q, bd, w.s, vd, 0.0, None, None, d, dd, self.space.desc)

    def __call__(self, x, ids, weights):
        """x: tokens x H bfloat16; ids, weights: tokens x top_k (each token's experts and their shares)."""
        ids, weights = ids.int().contiguous(), weights.float().contiguous()
        self.engine.group_rows(self.experts, ids, qg.layout("i32", self.tokens, self.top_k), self.offsets, self.rows, self.back,
                               self.space.desc)
        self.x.fill(self.engine, x, rows=self.rows)
        self.product(self.x, self.w1, self.gate_up, self.offsets)
        self.h.fill(self.engine, self.gate_up, act=qg.MX_SWIGLU)
        self.product(self.h, self.w2, self.out, self.offsets)
        y = torch.empty(self.tokens, self.hidden, device="cuda")
        self.engine.combine(self.out, qg.layout("bf16", *self.out.shape), self.back, weights, qg.layout("f32", self.tokens, self.top_k),
                            y, qg.layout("f32", self.tokens, self.hidden))
        return y


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    a = ap.parse_args()
    torch.manual_seed(0)
    engine = qg.Gemm()
    w1 = torch.randn(a.experts, 2 * a.inner, a.hidden, device="cuda", dtype=torch.bfloat16) * 0.02
    w2 = torch.randn(a.experts, a.hidden, a.inner, device="cuda", dtype=torch.bfloat16) * 0.02
    block = ExpertBlock(engine, w1, w2, a.tokens, a.top_k)
    x = torch.randn(a.tokens, a.hidden, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(a.tokens, -(-a.experts // 4) * 4, device="cuda")
    ids, share = torch.empty(a.tokens, a.top_k, device="cuda", dtype=torch.int32), torch.empty(a.tokens, a.top_k, device="cuda")
    engine.route(qg.routing(qg.ROUTE_SOFTMAX, a.top_k, renormalize=True), logits, qg.layout("f32", a.tokens, a.experts, ld=logits.shape[1]),
                 None, ids, qg.layout("i32", a.tokens, a.top_k), share, qg.layout("f32", a.tokens, a.top_k))
    for _ in range(3):
        y = block(x, ids, share)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        y = block(x, ids, share)
    end.record()
    torch.cuda.synchronize()
    flop = 6 * a.tokens * a.top_k * a.hidden * a.inner
    ms = begin.elapsed_time(end) / 10
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, {a.top_k} each: {ms:.3f} ms, "
          f"{flop / ms / 1e9:.0f} TFLOP/s, output rms {y.pow(2).mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
