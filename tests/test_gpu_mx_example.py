"""The MXFP4 operators together: an expert block, each step against the step in 64 bits on what the step before left.
The quantising steps are exact. Products are off by fp32 sums (2^-24 (K + 2) of sum |a b|) and half a step of bfloat16
(2^-8), the last weighted sum of top_k values by fp32 (2^-24 (top_k + 1) of sum |w d|)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import quantized_gemm_bf16_amd as qg
from tests import mx_ref

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx_experts.py")
    spec = importlib.util.spec_from_file_location("mx_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def decoded(m, rows):
    return mx_ref.values(mx_ref.unpack(m.q.cpu().numpy()), m.s.cpu().numpy()[:, :-(-m.cols // 32)])[:rows, :m.cols]


def rounded(x):
    return mx_ref.values(*mx_ref.quantise(x))[:, :x.shape[1]]


def check_product(got, a, b, owner, experts):
    for e in range(experts):
        ref, ab = a[owner == e] @ b[e].T, np.abs(a[owner == e]) @ np.abs(b[e]).T
        tol = 2.0 ** -24 * (a.shape[1] + 2) * ab
        assert (np.abs(got[owner == e] - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all(), e


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inner", [(1, 4, 2, 64, 32), (37, 8, 3, 200, 72), (300, 16, 4, 512, 264)])
def test_expert_block(tokens, experts, top_k, hidden, inner):
    torch.manual_seed(tokens)
    w1 = torch.randn(experts, 2 * inner, hidden, dtype=torch.bfloat16) * 0.1
    w2 = torch.randn(experts, hidden, inner, dtype=torch.bfloat16) * 0.1
    x = torch.randn(tokens, hidden, dtype=torch.bfloat16)
    share, ids = torch.randn(tokens, experts).softmax(-1).topk(top_k, -1)
    block = example().ExpertBlock(qg.Gemm(), w1.cuda(), w2.cuda(), tokens, top_k)
    y = block(x.cuda(), ids.cuda(), share.cuda()).double().cpu().numpy()
    owner, order = ids.flatten().sort(stable=True)
    owner, order = owner.numpy(), order.numpy()
    a = rounded(x.double().numpy())[order // top_k]
    assert np.array_equal(decoded(block.x, len(order)), a)
    gate_up = block.gate_up.double().cpu().numpy()
    check_product(gate_up, a, [rounded(w.double().numpy()) for w in w1], owner, experts)
    h = rounded(mx_ref.swiglu(gate_up))
    assert np.array_equal(decoded(block.h, len(order)), h)
    out = block.out.double().cpu().numpy()
    check_product(out, h, [rounded(w.double().numpy()) for w in w2], owner, experts)
    want, size = np.zeros((2, tokens, hidden))
    part = out * share.flatten().double().numpy()[order][:, None]
    np.add.at(want, order // top_k, part)
    np.add.at(size, order // top_k, np.abs(part))
    assert (np.abs(y - want) <= 2.0 ** -24 * (top_k + 1) * size).all()


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inner", [(1, 4, 2, 64, 32), (300, 16, 4, 512, 264)])
def test_expert_block_in_a_graph(tokens, experts, top_k, hidden, inner):
    """Captured, the block gives what it gives eagerly, replay after replay, with other tokens and other experts chosen."""
    torch.manual_seed(7)

    def inputs():
        share, ids = torch.randn(tokens, experts, device="cuda").softmax(-1).topk(top_k, -1)
        return torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16), ids, share

    w1 = torch.randn(experts, 2 * inner, hidden, device="cuda", dtype=torch.bfloat16) * 0.1
    w2 = torch.randn(experts, hidden, inner, device="cuda", dtype=torch.bfloat16) * 0.1
    block = example().ExpertBlock(qg.Gemm(), w1, w2, tokens, top_k)
    held = inputs()
    block(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(*held)
    for _ in range(4):
        new = inputs()
        want = block(*new).clone()
        for t, n in zip(held, new):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
