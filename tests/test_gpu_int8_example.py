"""The operators of an int8 expert block together: each step against the step in 64 bits on what the step before left. Choice,
sorting and quantising are exact. A product's value takes three roundings of fp32 before half a step of bfloat16; the weighted sum
top_k + 1 of sum |w d| + |x|, and half a step."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_experts.py")
    spec = importlib.util.spec_from_file_location("int8_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def make(tokens, experts, groups, top_k, hidden, inner, seed):
    torch.manual_seed(seed)
    router = torch.randn(experts, hidden, dtype=torch.bfloat16) * 0.1
    bias = torch.randn(experts) * 0.05
    w1 = torch.randn(experts, 2 * inner, hidden, dtype=torch.bfloat16) * 0.1
    w2 = torch.randn(experts, hidden, inner, dtype=torch.bfloat16) * 0.1
    kw = dict(groups=groups, top_groups=max(1, groups // 2), group_best=2, renormalize=True, scale=1.5)
    block = example().ExpertBlock(qg.Gemm(), router.cuda(), bias.cuda(), w1.cuda(), w2.cuda(), tokens, qg.routing(qg.ROUTE_SIGMOID, top_k, **kw))
    return block, bias, w1, w2, kw


def check_codes(codes, y):
    q, s = ref.quantise(y)
    assert np.array_equal(codes.q.cpu().numpy()[:, :codes.cols], q) and np.array_equal(codes.s.cpu().numpy(), s)
    return q.astype(np.float64) * s[:, None].astype(np.float64)


def check_product(got, a, b, offsets, n):
    for e in range(len(offsets) - 1):
        rows = slice(offsets[e], offsets[e + 1])
        want = a[rows] @ b[e * n:(e + 1) * n].T
        tol = 3.01 * 2.0 ** -24 * np.abs(want)
        # (the sum itself is exact; `want` is off by 2^-53 of its terms)
        tol += 2.0 ** -52 * a.shape[1] * (np.abs(a[rows]) @ np.abs(b[e * n:(e + 1) * n].T))
        assert (np.abs(got[rows] - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all(), e


@pytest.mark.parametrize("tokens,experts,groups,top_k,hidden,inner", [(1, 8, 1, 2, 64, 32), (37, 16, 4, 3, 200, 72), (300, 24, 3, 4, 512, 264),
                                                                      (5000, 8, 2, 2, 64, 40)])
def test_expert_block(tokens, experts, groups, top_k, hidden, inner):
    block, bias, w1, w2, kw = make(tokens, experts, groups, top_k, hidden, inner, tokens)
    x = torch.randn(tokens, hidden, dtype=torch.bfloat16)
    y = block(x.cuda()).double().cpu().numpy()
    ids, w = block.ids.cpu().numpy().reshape(tokens, top_k), block.weights.cpu().numpy().reshape(tokens, top_k)
    logits = block.logits.double().cpu().numpy()
    want, ww = ref.route(logits, top_k, True, bias.double().numpy(), **kw)
    assert np.array_equal(ids, want)
    assert (np.abs(w - ww) <= (24 + 1.5 * np.abs(logits).max()) * 2.0 ** -23 * np.abs(ww)).all()
    offsets, rows, back = ref.group(ids, experts)
    assert np.array_equal(block.offsets.cpu().numpy(), offsets) and np.array_equal(block.rows.cpu().numpy(), rows)
    assert np.array_equal(block.back.cpu().numpy().reshape(back.shape), back)
    a = check_codes(block.x, x.double().numpy()[rows])
    b1 = check_codes(block.w1, w1.flatten(0, 1).double().numpy())
    b2 = check_codes(block.w2, w2.flatten(0, 1).double().numpy())
    gate_up = block.gate_up.double().cpu().numpy()
    check_product(gate_up, a, b1, offsets, 2 * inner)
    h = check_codes(block.h, ref.swiglu(gate_up))
    out = block.out.double().cpu().numpy()
    check_product(out, h, b2, offsets, hidden)
    part = out[back] * w[..., None].astype(np.float64)
    want = part.sum(1) + x.double().numpy()
    tol = (top_k + 1) * 2.0 ** -24 * (np.abs(part).sum(1) + np.abs(x.double().numpy()))
    assert (np.abs(y - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("tokens,experts,groups,top_k,hidden,inner", [(1, 8, 1, 2, 64, 32), (3000, 16, 4, 4, 128, 72)])
def test_expert_block_in_a_graph(tokens, experts, groups, top_k, hidden, inner):
    """Captured, the block gives what it gives eagerly, replay after replay, with other tokens and so other experts."""
    block = make(tokens, experts, groups, top_k, hidden, inner, 3)[0]

    def new():
        return torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16)

    held = new()
    block(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(held)
    for _ in range(4):
        x = new()
        want = block(x).clone()
        held.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_two_blocks_on_two_streams():
    """Each with its own workspace, at the same time: what each gives alone."""
    blocks = [make(2100, 16, 4, 4, 128, 72, s)[0] for s in (1, 2)]
    xs = [torch.randn(2100, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = [b(x).clone() for b, x in zip(blocks, xs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, b, x in zip(streams, blocks, xs):
            with torch.cuda.stream(s):
                got.append(b(x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
